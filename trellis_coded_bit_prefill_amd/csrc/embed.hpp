// Embedding from a packed vocabulary matrix with trained rows behind it, and the
// trained rows' gradient from rows sorted by token. Part of rows.hip.

namespace trellis {
namespace {

// A wave takes `pairs` pairs of 256-column blocks of one row, half of it a
// block: lane l of a half decodes columns 8 l .. +7, whose windows lie in 40
// bits of two words, and stores 16 bytes.
template <int BITS>
__global__ __launch_bounds__(256) void embed_kernel(const int32_t *__restrict__ tokens, int64_t waves, int per_row,
                                                    int pairs, int blocks, const uint32_t *__restrict__ codes,
                                                    const uint16_t *__restrict__ scales, int n, float scale,
                                                    const uint16_t *__restrict__ extra, int count,
                                                    uint16_t *__restrict__ out) {
  constexpr int wpb = 8 * BITS;
  const int64_t id = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (id >= waves) return;
  const int64_t row = id / per_row;
  const int lane = threadIdx.x & 31, b0 = (int)(id - row * per_row) * 2 * pairs + ((threadIdx.x >> 5) & 1);
  const int b1 = b0 + 2 * pairs < blocks ? b0 + 2 * pairs : blocks;
  const int token = __builtin_amdgcn_readfirstlane(tokens[row]);
  uint16_t *const o = out + row * blocks * 256 + 8 * lane;
  if (token >= 0 && token < n) {
    const uint32_t *const w = codes + (int64_t)token * blocks * wpb;
    const float s = bf16_bits_to_f32(scales[token]);
    float q, kq;
    alu_row_constants(s, q, kq);
    const bool chain = __builtin_amdgcn_readfirstlane(!alu_scale_ok(s)) != 0;
    const int pos = (248 - 8 * lane) * BITS, w0 = pos >> 5, w1 = w0 + 1 == wpb ? 0 : w0 + 1;
    auto decode = [&](auto chained) {
      for (int b = b0; b < b1; b += 2) {
        const uint32_t *const bw = w + b * wpb;
        const uint64_t f = (((uint64_t)bw[w1] << 32) | bw[w0]) >> (pos & 31);
        u32x4 v;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float e[2];
#pragma unroll
          for (int h = 0; h < 2; ++h)
            e[h] = (float)(__bf16)window_weight((uint32_t)(f >> ((7 - 2 * c - h) * BITS)) & 0xFFFu, s, q, kq, decltype(chained)::value) * scale;
          v[c] = (uint32_t)bf16_of(e[0]) | ((uint32_t)bf16_of(e[1]) << 16);
        }
        *reinterpret_cast<u32x4 *>(o + b * 256) = v;
      }
    };
    if (chain) decode(std::true_type{});  // (two loops: a choice at every weight costs more than the weight)
    else decode(std::false_type{});
    return;
  }
  const bool trained = token >= n && token - n < count;
  const uint16_t *const x = extra + (trained ? (int64_t)(token - n) * blocks * 256 + 8 * lane : 0);
  for (int b = b0; b < b1; b += 2) {
    u32x4 v = {0u, 0u, 0u, 0u};
    if (trained) {
      v = *reinterpret_cast<const u32x4 *>(x + b * 256);
#pragma unroll
      for (int c = 0; c < 4; ++c)
        v[c] = (uint32_t)bf16_of(bf16_half(v[c], 0) * scale) | ((uint32_t)bf16_of(bf16_half(v[c], 1) * scale) << 16);
    }
    *reinterpret_cast<u32x4 *>(o + b * 256) = v;
  }
}

constexpr int64_t kEmbedWaves = 1 << 25;  // of a launch

// ---- gradient: rows sorted by token -------------------------------------------
// A stable radix sort of (trained row, row of dout), eight bits a pass, each
// pass: digits counted by 2048 rows, the counts' running sums, the rows placed.
// The first pass leaves out the rows without a trained token.
constexpr int kSortRows = 2048;   // of a workgroup
constexpr int kSortWave = kSortRows / 4;

// The wave's LDS accesses before this come before those behind it, other lanes'
// too. (LDS keeps a wave's accesses in order; the fence keeps the compiler's: a
// wave barrier alone says nothing of memory.)
__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

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
    wave_order();
    if (in && (same >> lane) == 1ull) counts[wave][digit] += (uint32_t)__popcll(same);
    wave_order();
  }
}

// Up to 16384 rows in one launch. Each workgroup sorts the pairs of `width`
// trained rows: it looks at every token, counts those before its own, which is
// where its pairs begin, and no workgroup waits for another. 256 trained rows are
// one pass. 16384 rows of 16384 trained ones take 16.2 us with 64 workgroups and
// 28.6 with one; up to 1024 rows have only one (one pair a lane; at 509 rows of
// 16384 the call takes 17.2 and 19.1). Every lane keeps up to 16 pairs in
// registers, each wave's in a row of positions, and LDS takes them to their next
// places, the last ones too (stored to memory as they come, four bytes a line,
// they took 13 us of 32).
constexpr int kSmallRows = 16384;
constexpr int kSmallGroups = 64;   // workgroups at most
constexpr int kSmallWidth = 256;   // trained rows of a workgroup at least
constexpr int kRowBits = 14;
static_assert(1 << kRowBits == kSmallRows, "a pair's row");
constexpr int kMostWidth = 1 << (32 - kRowBits);
static_assert(TRELLIS_MAX_TRAINED / kSmallGroups <= kMostWidth, "a pair's trained row");
struct SmallSort {
  uint32_t pair[kSmallRows];  // trained row of the workgroup's << 14 | row of dout
  uint16_t counts[16][256];
  uint32_t waves[4];
  uint32_t total;
  int32_t below[16], own[16];
};
__global__ __launch_bounds__(1024) void sort_small_kernel(Sort S, int width, uint32_t *__restrict__ arrived, int counters) {
  extern __shared__ __attribute__((aligned(16))) unsigned char small_space[];
  SmallSort &M = *reinterpret_cast<SmallSort *>(small_space);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int i = (int)blockIdx.x * 1024 + tid; i < counters; i += (int)gridDim.x * 1024) arrived[i] = 0u;
  constexpr int kEach = kSmallRows / 1024;
  uint32_t pair[kEach];
  int rank[kEach];
  uint32_t in = 0, under = 0;  // bit i: pair i exists, is another workgroup's before this one
  const int low = (int)blockIdx.x * width, high = S.count - low < width ? S.count - low : width;
  int each = (S.m + 1023) >> 10, i0 = wave * (64 * each) + lane, begin = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int at = i0 + 64 * i, token = S.tokens[at < S.m ? at : S.m - 1];
    const bool there = i < each && at < S.m && token >= S.first && token - S.first < S.count;
    const int mine = there ? token - S.first - low : -1;
    const bool have = mine >= 0 && mine < high;
    pair[i] = have ? (uint32_t)mine << kRowBits | (uint32_t)at : 0u;
    in |= (uint32_t)have << i;
    under |= (uint32_t)(there && mine < 0) << i;
  }
  if (gridDim.x > 1) {
    // The workgroup's own pairs move together, in order.
    int own = 0, below = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      own += (int)__popcll(__ballot((in >> i) & 1));
      below += (int)__popcll(__ballot((under >> i) & 1));
    }
    if (lane == 0) {
      M.below[wave] = below;
      M.own[wave] = own;
    }
    __syncthreads();
    int at = 0, all = 0;
#pragma unroll
    for (int w = 0; w < 16; ++w) {
      begin += M.below[w];
      at += w < wave ? M.own[w] : 0;
      all += M.own[w];
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const bool have = (in >> i) & 1;
      const uint64_t some = __ballot(have);
      if (have) M.pair[at + (int)__popcll(some & ((1ull << lane) - 1ull))] = pair[i];
      at += (int)__popcll(some);
    }
    __syncthreads();
    each = (all + 1023) >> 10;
    i0 = wave * (64 * each) + lane;
    in = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int from = i0 + 64 * i;
      in |= (uint32_t)(i < each && from < all) << i;
      pair[i] = M.pair[from < kSmallRows ? from : 0];  // (past the last pair: not used)
    }
    __syncthreads();
  }
  // As few passes as 8 bits each allow, of as few bits as they need: every bit of
  // a digit costs six operations a pair.
  const int all = 32 - __builtin_clz((width - 1) | 1), passes = (all + 7) >> 3, bits = (all + passes - 1) / passes;
  const uint32_t mask = (1u << bits) - 1u;
  for (int shift = 0;; shift += bits) {
    for (int i = tid; i < 16 * 256; i += 1024) (&M.counts[0][0])[i] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const bool have = (in >> i) & 1;
      uint64_t same = __ballot(have);
      int place = 0;
      if (same) {
        const uint32_t digit = pair[i] >> (kRowBits + shift) & mask;
#pragma unroll
        for (int b = 0; b < 8; ++b)
          if (b < bits) {
            const uint64_t set = __ballot((digit >> b) & 1u);
            same &= (digit >> b) & 1u ? set : ~set;
          }
        const int before = M.counts[wave][digit];
        place = before + (int)__popcll(same & ((1ull << lane) - 1ull));
        wave_order();
        if (have && (same >> lane) == 1ull) M.counts[wave][digit] = (uint16_t)(before + (int)__popcll(same));
        wave_order();
      }
      rank[i] = place;
    }
    __syncthreads();
    // places of each digit's first pair of each wave: thread d < 256, digit d
    uint32_t own = 0, sum = 0;
    if (tid < 256) {
#pragma unroll
      for (int w = 0; w < 16; ++w) own += M.counts[w][tid];
      sum = own;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const uint32_t up = __shfl_up(sum, o);
        if (lane >= o) sum += up;
      }
      if (lane == 63) M.waves[wave] = sum;
    }
    __syncthreads();
    if (tid < 256) {
      uint32_t at = sum - own;
      for (int w = 0; w < wave; ++w) at += M.waves[w];
      if (tid == 255) M.total = at + own;
#pragma unroll
      for (int w = 0; w < 16; ++w) {
        const uint32_t c = M.counts[w][tid];
        M.counts[w][tid] = (uint16_t)at;
        at += c;
      }
    }
    __syncthreads();
    const bool last = shift + bits >= all;
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if ((in >> i) & 1) M.pair[M.counts[wave][pair[i] >> (kRowBits + shift) & mask] + rank[i]] = pair[i];
    __syncthreads();
    if (last) break;
    in = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int at = i0 + 64 * i;
      in |= (uint32_t)(i < each && at < (int)M.total) << i;
      pair[i] = M.pair[at < kSmallRows ? at : 0];
    }
    __syncthreads();
  }
  for (int i = tid; i < (int)M.total; i += 1024) {
    S.key_out[begin + i] = low + (int)(M.pair[i] >> kRowBits);
    S.row_out[begin + i] = (int)(M.pair[i] & (kSmallRows - 1));
  }
  if (tid == 0 && blockIdx.x == gridDim.x - 1) *S.total = (uint32_t)begin + M.total;
}

// Sums of the sorted rows: a wave takes one chunk of pairs and 512 columns (8 a
// lane), and adds up the runs of equal tokens. A run that lies within the chunk
// is finished; what the chunk holds of one that goes on before or behind it goes
// to `parts`, and the wave that arrives last at the run adds its parts in order,
// of a long run those of 32 neighbouring chunks first, then their sums (16384
// equal tokens: 45 us a call against 118 with all parts added by one wave).
// The workgroups behind those write zeros in the trained rows that no pair
// names: a wave a row, which looks its token up in the sorted pairs.
constexpr int kChunkGroup = 32;
struct Sums {
  const uint16_t *dout;
  const int32_t *key, *row;
  const uint32_t *total;
  uint16_t *dextra;
  float *parts;       // [chunks][2][k]: of the chunk's first run, of its last
  // Zero. [chunks][column blocks], of the run that begins in the chunk and goes on
  // behind it: the chunks of its first group that arrived, and << 16 the groups;
  // then [groups][column blocks], the chunks of the run that comes into the group.
  // (The lower half counts to 64 at most.)
  uint32_t *arrived;
  int32_t k, chunk, chunks, count, columns;  // columns: blocks of 512
  float scale;
};
__device__ __forceinline__ void store8(uint16_t *p, const float (&v)[8], float scale) {
  u32x4 o;
#pragma unroll
  for (int e = 0; e < 4; ++e) o[e] = (uint32_t)bf16_of(v[2 * e] * scale) | ((uint32_t)bf16_of(v[2 * e + 1] * scale) << 16);
  __builtin_nontemporal_store(o, reinterpret_cast<u32x4 *>(p));
}
// Whether a pair has this key: the wave looks at 64 places at a time.
__device__ __forceinline__ bool find_pair(const int32_t *keys, int total, int key, int lane) {
  int low = 0, high = total;  // the first pair whose key is not below `key` lies in low .. high
  while (low < high) {
    const int step = (high - low + 63) >> 6, at = low + lane * step;
    const int k = at < high ? keys[at] : 0x7fffffff;
    if (__any(k == key)) return true;
    const int below = (int)__popcll(__ballot(k < key));
    if (step == 1) return false;
    const int next = low + below * step;
    high = next < high ? next : high;
    low += below > 0 ? (below - 1) * step + 1 : 0;
    if (below == 0) return false;
  }
  return false;
}
__global__ __launch_bounds__(64) void sum_runs_kernel(Sums S) {
  const int total = (int)*S.total, lane = threadIdx.x;
  if ((int)blockIdx.x >= S.chunks * S.columns) {
    const int e = (int)blockIdx.x - S.chunks * S.columns;
    if (find_pair(S.key, total, e, lane)) return;
    for (int c = 8 * lane; c < S.k; c += 512)
      __builtin_nontemporal_store(u32x4{0u, 0u, 0u, 0u}, reinterpret_cast<u32x4 *>(S.dextra + (int64_t)e * S.k + c));
    return;
  }
  const int chunk = (int)blockIdx.x / S.columns, column = (int)blockIdx.x - chunk * S.columns;
  const int c = column * 512 + 8 * lane;
  const bool mine = c < S.k;  // (the last block may be half a wave's)
  const int begin = chunk * S.chunk, end = total - begin < S.chunk ? total : begin + S.chunk;
  if (begin >= end) return;
  const int before_key = begin > 0 ? S.key[begin - 1] : -1, behind_key = end < total ? S.key[end] : -1;
  const __amdgpu_buffer_rsrc_t ws =
      __builtin_amdgcn_make_buffer_rsrc(S.parts, (short)0, (int)((uint32_t)S.chunks * 2u * (uint32_t)S.k * 4u), kRawBuffer);
  auto part_at = [&](int chunk, int which) { return ((uint32_t)(chunk * 2 + which) * (uint32_t)S.k + (uint32_t)c) * 4u; };
  float acc[8] = {};
  int key = -1, run = begin, shared[2] = {-1, -1};
  auto flush = [&](int next) {
    const bool before = run == begin && before_key == key, behind = next == end && behind_key == key;
    if (before || behind) {
      shared[before ? 0 : 1] = key;  // (a run that fills the chunk and goes on to both sides is its first)
      if (mine) {
#pragma unroll
        for (int e = 0; e < 8; e += 4)
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, f32x4{acc[e], acc[e + 1], acc[e + 2], acc[e + 3]}),
                                                 ws, part_at(chunk, before ? 0 : 1) + 4u * e, 0, kSc1);
      }
    } else if (mine) {
      store8(S.dextra + (int64_t)key * S.k + c, acc, S.scale);
    }
    run = next;
  };
  for (int i0 = begin; i0 < end; i0 += 64) {
    // 64 pairs, one a lane, and their rows eight at a time
    const int n = end - i0 < 64 ? end - i0 : 64;
    const int at = i0 + (lane < n ? lane : n - 1);
    const int keys = S.key[at], rows = S.row[at];
    constexpr int U = 8;
    for (int i = 0; i < n; i += U) {
      u32x4 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = __builtin_amdgcn_readlane(rows, i + u < n ? i + u : n - 1);
        v[u] = u32x4{0u, 0u, 0u, 0u};
        if (mine) v[u] = *reinterpret_cast<const u32x4 *>(S.dout + (int64_t)r * S.k + c);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (i + u >= n) break;
        const int next = __builtin_amdgcn_readlane(keys, i + u);
        if (next != key) {
          if (key >= 0) flush(i0 + i + u);
          key = next;
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[e] = 0.f;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] += bf16_half(v[u][e >> 1], e & 1);
      }
    }
  }
  flush(end);
  // Runs over several chunks: the parts are complete at the coherent level
  // before the count moves.
  if (shared[0] < 0 && shared[1] < 0) return;
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll 1
  for (int i = 0; i < 2; ++i) {
    const int whose = i ? shared[1] : shared[0];
    if (whose < 0) continue;
    // The run's chunks: the borders on both sides that it goes over, 64 at a time.
    int c0 = chunk, c1 = chunk;
    for (;;) {
      const int border = c0 - lane;
      const uint64_t over = __ballot(border > 0 && S.key[border > 0 ? (int64_t)border * S.chunk - 1 : 0] == whose);
      c0 -= over == ~0ull ? 64 : __builtin_ctzll(~over);
      if (over != ~0ull) break;
    }
    for (;;) {
      const int64_t border = (int64_t)(c1 + 1 + lane) * S.chunk;
      const uint64_t over = __ballot(border < total && S.key[border < total ? border : 0] == whose);
      c1 += over == ~0ull ? 64 : __builtin_ctzll(~over);
      if (over != ~0ull) break;
    }
    // The parts of the run's chunks in this group of chunks, and by the last of
    // these waves, where the run has chunks in several groups, the groups' sums
    // (up to 64 chunks: all its parts at once, as a second round takes 2 us more).
    // (A run's first chunk keeps its part as the last run's, the others as the
    // first's; a group's sum stands in place of its first part. Past the last
    // chunk: outside the buffer, zero.)
    auto arrive = [&](uint32_t *count, uint32_t one) {
      uint32_t was = 0;
      if (lane == 0) was = __hip_atomic_fetch_add(count, one, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      return (uint32_t)__builtin_amdgcn_readfirstlane(was);
    };
    const bool one = c1 - c0 < 2 * kChunkGroup;
    const int group = chunk / kChunkGroup, g0 = c0 / kChunkGroup, groups = one ? 1 : c1 / kChunkGroup - g0 + 1;
    const int from = one || group == g0 ? c0 : group * kChunkGroup;
    const int to = one || group == c1 / kChunkGroup ? c1 : (group + 1) * kChunkGroup - 1;
    uint32_t *const begins = S.arrived + (int64_t)c0 * S.columns + column;
    uint32_t *const comes = S.arrived + ((int64_t)S.chunks + group) * S.columns + column;
    if ((arrive(from > c0 ? comes : begins, 1u) & 0xFFFFu) != (uint32_t)(to - from)) continue;
    int at = from, step = 1, n = to - from + 1;
    bool done;
#pragma unroll 1
    for (;;) {
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = 0.f;
      constexpr int U = 8;
#pragma unroll 1
      for (int j = 0; j < n; j += U) {
        f32x4 v[U][2];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int p = j + u == 0 && at < c0 ? c0 : at + (j + u) * step;
            v[u][h] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                    ws, mine && j + u < n ? part_at(p, p == c0) + 16u * h : 0xFFFFFFF0u, 0, kSc1));
          }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[e] += v[u][e >> 2][e & 3];
      }
      done = step > 1 || groups == 1;
      if (done) break;
      if (mine) {
#pragma unroll
        for (int e = 0; e < 8; e += 4)
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, f32x4{acc[e], acc[e + 1], acc[e + 2], acc[e + 3]}),
                                                 ws, part_at(from, from == c0) + 4u * e, 0, kSc1);
      }
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      if (arrive(begins, 1u << 16) >> 16 != (uint32_t)(groups - 1)) break;
      at = g0 * kChunkGroup;  // (the first group's sum stands at c0)
      step = kChunkGroup;
      n = groups;
    }
    if (!done) continue;
    if (mine) store8(S.dextra + (int64_t)whose * S.k + c, acc, S.scale);
  }
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
  // One pair of blocks a wave until the card is full (8192 waves), then up to
  // four, which share the token's and the scale's loads; more only for outputs
  // beyond 128 GiB (a launch has fewer than 2^32 threads).
  const int both = (blocks + 1) / 2;
  int pairs = (int)((int64_t)m * both / 8192);
  pairs = pairs < 1 ? 1 : pairs > 4 ? 4 : pairs;
  while ((int64_t)m * ((both + pairs - 1) / pairs) > kEmbedWaves) pairs *= 2;
  const int per_row = (both + pairs - 1) / pairs;
  const int64_t waves = (int64_t)m * per_row;
  const dim3 grid((unsigned)((waves + 3) / 4));
  (void)hipGetLastError();
  const auto fn = g.bits == 2 ? &embed_kernel<2> : g.bits == 3 ? &embed_kernel<3> : &embed_kernel<4>;
  hipLaunchKernelGGL(fn, grid, dim3(256), 0, stream, tokens, waves, per_row, pairs, blocks, codes, scales, g.n, scale, extra, count, out);
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
  // Chunks of 16 pairs at least; at most 1024 chunks and 2 GiB of parts.
  int64_t most = ((int64_t)1 << 31) / ((int64_t)k * 8);
  if (most > 1024) most = 1024;
  int chunk = (int)((m + most - 1) / most);
  if (chunk < 16) chunk = 16;
  const int chunks = (m + chunk - 1) / chunk, columns = (k + 511) / 512;
  const int counters = (chunks + (chunks + kChunkGroup - 1) / kChunkGroup) * columns;
  const size_t pair_bytes = up256((size_t)m * 4), count_bytes = up256((size_t)blocks * 1024),
               part_bytes = (size_t)chunks * 2 * k * 4, arrived_bytes = up256((size_t)counters * 4);
  Space *w = nullptr;
  TRELLIS_TRY(space(dev, stream, 4 * pair_bytes + count_bytes + 256 + arrived_bytes + part_bytes, 0, w));
  unsigned char *at = w->bytes;
  auto take = [&](size_t bytes) {
    unsigned char *const p = at;
    at += bytes;
    return p;
  };
  int32_t *pairs[4];
  for (auto &p : pairs) p = reinterpret_cast<int32_t *>(take(pair_bytes));
  uint32_t *const counts = reinterpret_cast<uint32_t *>(take(count_bytes)), *const total = reinterpret_cast<uint32_t *>(take(256)),
           *const arrived = reinterpret_cast<uint32_t *>(take(arrived_bytes));
  float *const parts = reinterpret_cast<float *>(take(part_bytes));
  (void)hipGetLastError();
  int to = 0;
  if (m <= kSmallRows) {
    static bool ready[kMaxDevices];
    if (!ready[dev] && !worked(hipFuncSetAttribute(reinterpret_cast<const void *>(&sort_small_kernel),
                                                   hipFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(SmallSort))))
      return TRELLIS_E_HIP;
    ready[dev] = true;
    const Sort s{tokens, nullptr, nullptr, pairs[0], pairs[1], nullptr, total, m, first, count, 0, 0};
    int width = (count + kSmallGroups - 1) / kSmallGroups;
    if (width < kSmallWidth) width = kSmallWidth;
    if (count < width || (m <= 1024 && count <= kMostWidth)) width = count;
    hipLaunchKernelGGL(sort_small_kernel, dim3((unsigned)((count + width - 1) / width)), dim3(1024), sizeof(SmallSort), stream, s,
                       width, arrived, counters);
  } else {
    hipLaunchKernelGGL(clear_kernel, dim3((unsigned)((counters + 255) / 256)), dim3(256), 0, stream, arrived,
                       (int64_t)counters);
    for (int shift = 0; shift == 0 || (count - 1) >> shift; shift += 8, to ^= 2) {
      const Sort s{shift ? nullptr : tokens, pairs[to ^ 2], pairs[(to ^ 2) + 1], pairs[to], pairs[to + 1], counts, total, m,
                   first, count, shift, blocks};
      hipLaunchKernelGGL(sort_count_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, s);
      hipLaunchKernelGGL(sort_sum_kernel, dim3(1), dim3(1024), 0, stream, counts, 256 * blocks, total);
      hipLaunchKernelGGL(sort_place_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, s, total);
    }
    to ^= 2;  // the last pass's output
  }
  const Sums s{dout, pairs[to], pairs[to + 1], total, dextra, parts, arrived, k, chunk, chunks, count, columns, scale};
  hipLaunchKernelGGL(sum_runs_kernel, dim3((unsigned)(chunks * columns + count)), dim3(64), 0, stream, s);
  return hipGetLastError() == hipSuccess ? TRELLIS_OK : TRELLIS_E_HIP;
}

}  // extern "C"
