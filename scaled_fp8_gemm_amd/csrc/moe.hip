// moe.hip -- tokens sorted by expert and back, with their gradients.
//
// n = tokens * k choices, choice i = t * k + j of token t naming an expert.
//   counts[e]   choices of expert e (ids outside [0, experts) are dropped)
//   offsets     exclusive sums of counts rounded up to `pad`
//   pos[i]      offsets[e] + the number of earlier choices of e; -1 dropped
//   src         its inverse over the sorted rows; -1 in the padding
//   dispatch    xs[pos[i]] = x[t], padding rows inside segments zero
//   combine     y[t] = sum_j w[t][j] ys[pos[t][j]]
//   its gradient  dys[pos[t][j]] = w[t][j] dy[t], dw[t][j] = dy[t] . ys[pos[t][j]]
// (dispatch's gradient is combine without weights.)  The sort is a counting
// sort of the ids alone; the rest is bound by HBM and goes by token, so a
// token's row is read once however many experts take it.
// Measured (one MI355X, us):
//   sort of 16384 choices to 8 experts                  7.4  (16 tokens: 5.0)
//   sort of 131072 choices to 128 experts              14.5
//   sort of 10^6 choices to 128 / 1000 experts        104 / 784
//   dispatch, 8192 tokens x 4096, k 2, blockwise cast  33.5  4.1 TB/s
//   combine, 4096 tokens x 4096, k 6                   39.8  5.9 TB/s
//   its gradient, 8192 tokens x 5120, k 2              82    5.1 TB/s
// Beyond kSelfCount choices every workgroup of the sort adds up all
// workgroups' counts, which is what 10^6 choices spend their time on.
#include "tile.h"

namespace fp8sg {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kGroups = kThreads / 16;
constexpr int kSortThreads = 1024;             // also the choices ranked at a time
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kCounters = 8192;                // LDS counters, several per expert
constexpr int kMaxSortBlocks = 1024;
// Up to this many choices every workgroup counts all of them itself, which
// saves a launch; beyond, a first launch counts.  us, without and with the
// first launch: 16384 choices to 8 experts 7.8 and 11.0, 65536 to 8 11.0 and
// 11.1, 65536 to 1024 13.0 and 33.9, 131072 to 8 16.3 and 10.6, 131072 to 128
// 16.9 and 14.5.
constexpr int64_t kSelfCount = 65536;

// Counters per expert (a power of two, 8 .. 64), so that the lanes of a wave
// rarely add to one word.
__device__ __forceinline__ int counter_columns(int experts) {
  int c = 64;
  while (c * experts > kCounters) c >>= 1;
  return c;
}
__device__ __forceinline__ void count_choices(const int32_t* __restrict__ expert, int64_t from,
                                              int64_t to, int experts, int columns,
                                              uint32_t* counters) {
  const int col = threadIdx.x & (columns - 1);
  constexpr int U = 8;                         // loads in flight
  for (int64_t i = from + threadIdx.x; i < to; i += U * kSortThreads) {
    uint32_t e[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t at = i + u * kSortThreads;
      e[u] = at < to ? (uint32_t)expert[at] : 0xffffffffu;
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (e[u] < (uint32_t)experts) atomicAdd(&counters[e[u] * columns + col], 1u);
  }
}
// Counters -> counts; every thread sums 8 counters of one expert.
__device__ __forceinline__ void sum_counters(const uint32_t* counters, int experts, int columns,
                                             int32_t* counts) {
  const int at = threadIdx.x * 8, e = at / columns;
  uint32_t s = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) s += counters[at + i];
  for (int off = 1; off < columns / 8; off <<= 1) s += (uint32_t)__shfl_xor((int)s, off, 64);
  if (at % columns == 0 && e < experts) counts[e] = (int32_t)s;
}

__global__ __launch_bounds__(kSortThreads) void k_moe_count(const int32_t* __restrict__ expert,
                                                            int64_t n, int64_t chunk, int experts,
                                                            uint32_t* __restrict__ ws) {
  __shared__ uint32_t counters[kCounters];
  __shared__ int32_t counts[kMaxExperts];
  const int columns = counter_columns(experts);
  for (int i = threadIdx.x; i < kCounters; i += kSortThreads) counters[i] = 0;
  __syncthreads();
  const int64_t from = blockIdx.x * chunk, to = min(n, from + chunk);
  count_choices(expert, from, to, experts, columns, counters);
  __syncthreads();
  sum_counters(counters, experts, columns, counts);
  __syncthreads();
  for (int e = threadIdx.x; e < experts; e += kSortThreads)
    ws[(int64_t)blockIdx.x * experts + e] = (uint32_t)counts[e];
}

// Workgroup b places the choices [b * chunk, (b + 1) * chunk), 1024 at a
// time: a wave finds each lane's equals with one ballot per bit of the id,
// a lane's rank among them is the number of lower ones, and the waves'
// counts are added up in order.  SELF: counts everything itself.
template <bool SELF>
__global__ __launch_bounds__(kSortThreads) void k_moe_sort(
    const int32_t* __restrict__ expert, int64_t n, int64_t chunk, int experts, int pad,
    int64_t rows, const uint32_t* __restrict__ ws, int32_t* __restrict__ offsets,
    int32_t* __restrict__ counts, int32_t* __restrict__ pos, int32_t* __restrict__ src) {
  __shared__ uint32_t counters[kCounters];     // then the waves' counts (16-bit, [wave][expert])
  __shared__ int32_t before[kMaxExperts], total[kMaxExperts], start[kMaxExperts + 1];
  __shared__ int32_t wave_end[kSortWaves];
  static_assert(kSortWaves * kMaxExperts * 2 <= kCounters * 4, "the waves' counts");
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int64_t from = blockIdx.x * chunk, to = min(n, from + chunk);
  if constexpr (SELF) {
    const int columns = counter_columns(experts);
    for (int i = t; i < kCounters; i += kSortThreads) counters[i] = 0;
    __syncthreads();
    count_choices(expert, 0, from, experts, columns, counters);
    __syncthreads();
    sum_counters(counters, experts, columns, before);
    __syncthreads();
    count_choices(expert, from, n, experts, columns, counters);
    __syncthreads();
    sum_counters(counters, experts, columns, total);
  } else {
    for (int e = t; e < experts; e += kSortThreads) before[e] = total[e] = 0;
    __syncthreads();
    const int64_t all = (int64_t)gridDim.x * experts, mine = (int64_t)blockIdx.x * experts;
    for (int64_t i = t; i < all; i += kSortThreads) {
      const int32_t v = (int32_t)ws[i];
      const int e = (int)(i % experts);
      if (v) {
        atomicAdd(&total[e], v);
        if (i < mine) atomicAdd(&before[e], v);
      }
    }
  }
  __syncthreads();
  // offsets: exclusive sums of the padded counts, one expert per thread
  {
    const int32_t c = t < experts ? total[t] : 0;
    const int32_t padded = (int32_t)(((int64_t)c + pad - 1) / pad * pad);
    int32_t s = padded;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int32_t o = __shfl_up(s, off, 64);
      if (lane >= off) s += o;
    }
    if (lane == 63) wave_end[wave] = s;
    __syncthreads();
    for (int w = 0; w < wave; ++w) s += wave_end[w];
    if (t < experts) {
      start[t] = s - padded;
      if (t == experts - 1) start[experts] = s;
    }
  }
  __syncthreads();
  if (blockIdx.x == 0) {
    for (int e = t; e <= experts; e += kSortThreads) {
      offsets[e] = start[e];
      if (e < experts) counts[e] = total[e];
    }
  }
  // the padding of every segment, and the rows past the last
  for (int e = blockIdx.x * kSortWaves + wave; e < experts; e += gridDim.x * kSortWaves)
    for (int64_t r = (int64_t)start[e] + total[e] + lane; r < start[e + 1]; r += 64) src[r] = -1;
  for (int64_t r = (int64_t)start[experts] + (int64_t)blockIdx.x * kSortThreads + t; r < rows;
       r += (int64_t)gridDim.x * kSortThreads)
    src[r] = -1;

  uint16_t* wc = reinterpret_cast<uint16_t*>(counters);
  const int bits = 32 - __builtin_clz((uint32_t)experts);
  for (int64_t at = from; at < to; at += kSortThreads) {
    for (int i = t; i < kSortWaves * experts; i += kSortThreads) wc[i] = 0;
    __syncthreads();
    const int64_t i = at + t;
    const uint32_t id = i < to ? (uint32_t)expert[i] : 0xffffffffu;
    const bool kept = id < (uint32_t)experts;
    const int e = kept ? (int)id : 0;
    uint64_t same = __ballot(kept);
    for (int b = 0; b < bits; ++b) {
      const bool bit = (e >> b) & 1;
      const uint64_t m = __ballot(bit);
      same &= bit ? m : ~m;
    }
    const int rank = __popcll(same & ((1ull << lane) - 1));
    if (kept && rank == 0) wc[wave * experts + e] = (uint16_t)__popcll(same);
    __syncthreads();
    int32_t sum = 0;
    if (t < experts) {
#pragma unroll
      for (int w = 0; w < kSortWaves; ++w) {
        const int32_t c = wc[w * experts + t];
        wc[w * experts + t] = (uint16_t)sum;
        sum += c;
      }
    }
    __syncthreads();
    if (i < to) {
      const int32_t p = kept ? start[e] + before[e] + wc[wave * experts + e] + rank : -1;
      pos[i] = p;
      if (kept) src[p] = (int32_t)i;
    }
    __syncthreads();
    if (t < experts) before[t] += sum;
    // the next round's first barrier orders this before its reads
  }
}

// Zeros for the padding rows inside segments, `share` (at most 16) rows per
// workgroup: few in a small batch, where padding is most of the rows and
// nothing else runs, 16 where most workgroups find none.  us of dispatch with
// 1 and 16 (rows of 4096 columns): 144 rows 3.3 and 8.0, 1920 rows 8.5 and
// 10.3, 17280 rows with a cast 52 and 37.
int pad_share(int64_t rows) { return rows <= 1024 ? 1 : 16; }
__device__ __forceinline__ void zero_padding(const MoeRows& p, int64_t block, int64_t blocks,
                                             int share, uint16_t* xs, const CastOut& xq) {
  const int64_t end = min((int64_t)*p.end, p.rows);
  const float zero[8] = {};
  const int slots = (int)((p.cols + 7) >> 3);
  const int at = threadIdx.x & 15;
  for (int64_t first = block * share; first < end; first += blocks * share) {
    // one load finds all of the padding rows among these
    uint32_t todo = (uint32_t)__ballot(at < share && first + at < end && p.src[first + at] < 0) &
                    0xffffu;
    for (; todo; todo &= todo - 1) {
      const int64_t r = first + __builtin_ctz(todo);
      for (int slot = threadIdx.x; slot < slots; slot += kThreads) {
        const int64_t left = p.cols - (int64_t)slot * 8;
        const int nv = left < 8 ? (int)left : 8;
        if (xs) store_bf16x8(xs + r * p.cols + (int64_t)slot * 8, zero, nv, p.stream);
        if (xq.q) {
          SlotCast c;
          c.q = make_uint2(0, 0);
          if (xq.scaling == kCastMX) c.e8m0 = 127u;
          else c.scale_inv = 1.0f;
          store_cast(xq, c, r, p.cols, slot, nv);
        }
      }
    }
  }
}

// A wave takes K slots a lane of a token's row, all loaded before the first
// is cast; blockIdx.y walks the row's shares.  (By 16-lane groups of one slot
// each: 42.3 us at 8192 tokens x 4096, against 33.)
template <int K, bool TINY>
__global__ __launch_bounds__(kThreads) void k_moe_dispatch(const MoeRows p, int64_t token_blocks,
                                                           int share,
                                                           const uint16_t* __restrict__ x,
                                                           uint16_t* __restrict__ xs, CastOut xq) {
  if (blockIdx.x >= token_blocks) {
    if (blockIdx.y == 0)
      zero_padding(p, blockIdx.x - token_blocks, gridDim.x - token_blocks, share, xs, xq);
    return;
  }
  const float ts = xq.scaling == kCastTensor ? *xq.scale : 1.0f;
  const int lane = threadIdx.x & 63;
  for (int64_t tok = (int64_t)blockIdx.x * kWaves +
                     __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
       tok < p.tokens; tok += token_blocks * kWaves) {
    for (int64_t base = (int64_t)blockIdx.y * (K * 512); base < p.cols;
         base += (int64_t)gridDim.y * (K * 512)) {
      Slot<kInBF16> v[K];
      SlotCast c[K];
#pragma unroll
      for (int i = 0; i < K; ++i)
        v[i].template load<TINY>(x + tok * p.cols, base + i * 512 + lane * 8, p.cols);
#pragma unroll
      for (int i = 0; i < K; ++i) v[i].template settle<TINY>(base + i * 512 + lane * 8, p.cols);
      if (xq.q) {
        float f[K][8];
#pragma unroll
        for (int i = 0; i < K; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) f[i][e] = v[i].get(e);
        cast_slots<K>(xq.scaling, xq.fmt, f, ts, c);
      }
      for (int j = 0; j < p.k; ++j) {
        const int64_t r = (uint32_t)p.pos[tok * p.k + j];
        if (r >= p.rows) continue;
#pragma unroll
        for (int i = 0; i < K; ++i) {
          const int64_t col = base + i * 512 + lane * 8;
          const int64_t left = p.cols - col;
          const int nv = left < 8 ? (int)left : 8;
          if (xs && nv > 0) store_slot(xs + r * p.cols + col, v[i], nv);
          if (xq.q) store_cast(xq, c[i], r, p.cols, (int)(col >> 3), nv);
        }
      }
    }
  }
}

// KJ choices at a time: their loads go out together, a dropped one's from
// row 0 with its values put to zero (its row may hold anything).
template <int KJ, bool TINY>
__global__ __launch_bounds__(kThreads) void k_moe_combine(const MoeRows p,
                                                          const uint16_t* __restrict__ ys,
                                                          const float* __restrict__ weight,
                                                          uint16_t* __restrict__ y) {
  const int lane = threadIdx.x & 15;
  TileWalk w((int64_t)blockIdx.x * kGroups + (threadIdx.x >> 4), (int64_t)gridDim.x * kGroups,
             (int)((p.cols + 127) >> 7));
  for (; w.row < p.tokens; w.next()) {
    const int64_t col = (int64_t)w.tile * 128 + lane * 8;
    const int64_t left = p.cols - col;
    const int nv = left < 8 ? (int)left : 8;
    if (nv <= 0) continue;
    float acc[8] = {};
    for (int j0 = 0; j0 < p.k; j0 += KJ) {
      Slot<kInBF16> v[KJ];
      float wt[KJ];
      bool ok[KJ];
#pragma unroll
      for (int j = 0; j < KJ; ++j) {
        const int64_t c = w.row * p.k + min(j0 + j, p.k - 1);
        const int64_t r = (uint32_t)p.pos[c];
        ok[j] = r < p.rows && j0 + j < p.k;
        wt[j] = weight ? weight[c] : 1.0f;
        v[j].template load<TINY>(ys + (ok[j] ? r : 0) * p.cols, col, p.cols);
      }
#pragma unroll
      for (int j = 0; j < KJ; ++j) v[j].template settle<TINY>(col, p.cols);
#pragma unroll
      for (int j = 0; j < KJ; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = ok[j] ? acc[i] + wt[j] * v[j].get(i) : acc[i];
    }
    store_bf16x8(y + w.row * p.cols + col, acc, nv, p.stream);
  }
}

// Gradient of combine.  A token's threads (a wave, or the workgroup) walk
// its row once per KJ choices.
template <int KJ, bool WAVE, bool TINY>
__global__ __launch_bounds__(kThreads) void k_moe_combine_bwd(
    const MoeRows p, int64_t token_blocks, int share, const uint16_t* __restrict__ dy,
    const uint16_t* __restrict__ ys, const float* __restrict__ weight,
    uint16_t* __restrict__ dys, float* __restrict__ dw) {
  if (blockIdx.x >= token_blocks) {
    zero_padding(p, blockIdx.x - token_blocks, gridDim.x - token_blocks, share, dys, CastOut());
    return;
  }
  __shared__ float red[KJ][kThreads / 64];
  constexpr int nt = WAVE ? 64 : kThreads;
  const int t = threadIdx.x & (nt - 1);
  const int slots = (int)((p.cols + 7) >> 3);
  for (int64_t tok = WAVE ? (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6)
                          : (int64_t)blockIdx.x;
       tok < p.tokens; tok += token_blocks * (WAVE ? kWaves : 1)) {
    for (int j0 = 0; j0 < p.k; j0 += KJ) {
      float acc[KJ], wt[KJ];
      int64_t row[KJ];
      bool ok[KJ];
#pragma unroll
      for (int j = 0; j < KJ; ++j) {
        const int64_t c = tok * p.k + min(j0 + j, p.k - 1);
        const int64_t r = (uint32_t)p.pos[c];
        ok[j] = r < p.rows && j0 + j < p.k;
        row[j] = ok[j] ? r : 0;
        wt[j] = weight[c];
        acc[j] = 0.0f;
      }
      for (int slot = t; slot < slots; slot += nt) {
        const int64_t col = (int64_t)slot * 8;
        const int64_t left = p.cols - col;
        const int nv = left < 8 ? (int)left : 8;
        Slot<kInBF16> d, v[KJ];
        d.load<TINY>(dy + tok * p.cols, col, p.cols);
#pragma unroll
        for (int j = 0; j < KJ; ++j)
          v[j].template load<TINY>(ys + row[j] * p.cols, col, p.cols);
        d.settle<TINY>(col, p.cols);
#pragma unroll
        for (int j = 0; j < KJ; ++j) {
          v[j].template settle<TINY>(col, p.cols);
          if (!ok[j]) continue;
          float o[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            acc[j] += d.get(i) * v[j].get(i);
            o[i] = wt[j] * d.get(i);
          }
          store_bf16x8(dys + row[j] * p.cols + col, o, nv, p.stream);
        }
      }
#pragma unroll
      for (int j = 0; j < KJ; ++j) {
        acc[j] = wave_sum(acc[j]);
        if (!WAVE && (threadIdx.x & 63) == 0) red[j][threadIdx.x >> 6] = acc[j];
      }
      if constexpr (!WAVE) __syncthreads();
      if (t < KJ && j0 + t < p.k) {
        float s = 0.0f;
        bool live = false;
#pragma unroll
        for (int j = 0; j < KJ; ++j)
          if (j == t) {
            live = ok[j];
            s = acc[j];
          }
        if constexpr (!WAVE) s = red[t][0] + red[t][1] + red[t][2] + red[t][3];
        dw[tok * p.k + j0 + t] = live ? s : 0.0f;
      }
      if constexpr (!WAVE) __syncthreads();
    }
  }
}

int64_t sort_chunk(int64_t n) {
  const int64_t rounds = (n + (int64_t)kSortThreads * kMaxSortBlocks - 1) /
                         ((int64_t)kSortThreads * kMaxSortBlocks);
  return kSortThreads * (rounds > 1 ? rounds : 1);
}
int sort_blocks(int64_t n) {
  const int64_t c = sort_chunk(n);
  return n > 0 ? (int)((n + c - 1) / c) : 1;
}
int64_t at_most(int64_t n) { return n < kMaxGrid ? n : kMaxGrid; }
int64_t pad_blocks(int64_t rows) {
  return at_most((rows + pad_share(rows) - 1) / pad_share(rows));
}
int64_t tile_blocks(int64_t rows, int64_t cols) {
  const int64_t need = (rows * ((cols + 127) / 128) + kGroups - 1) / kGroups;
  return at_most(need);
}

}  // namespace

int64_t moe_workspace_words(int64_t n, int experts) { return (int64_t)sort_blocks(n) * experts; }

hipError_t launch_moe_sort(const int32_t* expert, int64_t n, int experts, int pad, int64_t rows,
                           int32_t* offsets, int32_t* counts, int32_t* pos, int32_t* src,
                           uint32_t* ws, hipStream_t s) {
  const int64_t chunk = sort_chunk(n);
  const int g = sort_blocks(n);
  if (n <= kSelfCount) {
    hipLaunchKernelGGL(k_moe_sort<true>, dim3(g), dim3(kSortThreads), 0, s, expert, n, chunk,
                       experts, pad, rows, ws, offsets, counts, pos, src);
  } else {
    hipLaunchKernelGGL(k_moe_count, dim3(g), dim3(kSortThreads), 0, s, expert, n, chunk, experts,
                       ws);
    hipLaunchKernelGGL(k_moe_sort<false>, dim3(g), dim3(kSortThreads), 0, s, expert, n, chunk,
                       experts, pad, rows, ws, offsets, counts, pos, src);
  }
  return hipGetLastError();
}

hipError_t launch_moe_dispatch(const MoeRows& p, const uint16_t* x, uint16_t* xs,
                               const CastOut& xq, hipStream_t s) {
  if (p.rows == 0 || p.cols == 0) return hipSuccess;
  const int share = pad_share(p.rows);
  const int64_t tb = at_most((p.tokens + kWaves - 1) / kWaves), gx = tb + pad_blocks(p.rows);
  // as many waves as there are slots / 64 while the chip runs them at once
  // (us with 1 and 2 slots a lane, rows of 4096: 16 tokens 3.3 and 3.9, 256
  // tokens 4.9 and 5.0, 8192 tokens with a cast 66 and 52 when each workgroup
  // looked for one padding row; 4 slots a lane: 33.0 against 33.1 at 8192)
  const int64_t shares = (p.cols + 511) / 512;
  const int k = shares == 1 || p.tokens * shares <= 4096 ? 1 : 2;
  const int64_t y = (shares + k - 1) / k;
  const dim3 grid((unsigned)gx, (unsigned)(y < 65535 ? y : 65535));
  if (p.cols < 8)
    hipLaunchKernelGGL((k_moe_dispatch<1, true>), grid, dim3(kThreads), 0, s, p, tb, share, x,
                       xs, xq);
  else if (k == 1)
    hipLaunchKernelGGL((k_moe_dispatch<1, false>), grid, dim3(kThreads), 0, s, p, tb, share, x,
                       xs, xq);
  else
    hipLaunchKernelGGL((k_moe_dispatch<2, false>), grid, dim3(kThreads), 0, s, p, tb, share, x,
                       xs, xq);
  return hipGetLastError();
}

#define FP8SG_K_DISPATCH(k, ...)                      \
  do {                                                \
    switch (k) {                                      \
      case 1: { constexpr int KJ = 1; __VA_ARGS__; } break; \
      case 2: { constexpr int KJ = 2; __VA_ARGS__; } break; \
      case 3: { constexpr int KJ = 3; __VA_ARGS__; } break; \
      case 4: { constexpr int KJ = 4; __VA_ARGS__; } break; \
      case 5: { constexpr int KJ = 5; __VA_ARGS__; } break; \
      case 6: { constexpr int KJ = 6; __VA_ARGS__; } break; \
      case 7: { constexpr int KJ = 7; __VA_ARGS__; } break; \
      default: { constexpr int KJ = 8; __VA_ARGS__; } break; \
    }                                                 \
  } while (0)

hipError_t launch_moe_combine(const MoeRows& rows, const uint16_t* ys, const float* weight,
                              uint16_t* y, hipStream_t s) {
  MoeRows p = rows;
  p.stream = 2 * p.cols * (p.tokens + p.tokens * p.k) > kStreamBytes;
  if (p.tokens * p.cols == 0) return hipSuccess;
  if (p.rows == 0) p.k = 0;                    // nothing to add up, or to read
  const int64_t g = tile_blocks(p.tokens, p.cols);
  if (p.cols < 8)
    hipLaunchKernelGGL((k_moe_combine<1, true>), dim3((unsigned)g), dim3(kThreads), 0, s, p, ys,
                       weight, y);
  else
    FP8SG_K_DISPATCH(p.k, hipLaunchKernelGGL((k_moe_combine<KJ, false>), dim3((unsigned)g),
                                             dim3(kThreads), 0, s, p, ys, weight, y));
  return hipGetLastError();
}

hipError_t launch_moe_combine_bwd(const MoeRows& rows, const uint16_t* dy, const uint16_t* ys,
                                  const float* weight, uint16_t* dys, float* dw, hipStream_t s) {
  MoeRows p = rows;
  p.stream = 2 * p.cols * (p.tokens + 2 * p.rows) > kStreamBytes;
  const int share = pad_share(p.rows);
  if (p.rows == 0) ys = dy;                    // all choices dropped: read, not used
  // a wave or a workgroup a token, us: 8192 x 520 14.0 and 21.0, 16384 x 1024
  // 34 and 42, 4096 x 8192 with k 1 42.5 and 45; but 8192 x 2048 43.5 and 32,
  // 8192 x 5120 82 and 77.5
  const bool wave = p.tokens >= 2048 || p.cols <= 512;
  const int64_t tb = at_most(wave ? (p.tokens + kWaves - 1) / kWaves : p.tokens);
  const int64_t g = tb + (p.cols > 0 ? pad_blocks(p.rows) : 0);
  if (g == 0) return hipSuccess;
  if (p.cols < 8) {
    hipLaunchKernelGGL((k_moe_combine_bwd<1, true, true>), dim3((unsigned)g), dim3(kThreads), 0, s,
                       p, tb, share, dy, ys, weight, dys, dw);
    return hipGetLastError();
  }
  FP8SG_K_DISPATCH(p.k, {
    if (wave)
      hipLaunchKernelGGL((k_moe_combine_bwd<KJ, true, false>), dim3((unsigned)g), dim3(kThreads), 0,
                         s, p, tb, share, dy, ys, weight, dys, dw);
    else
      hipLaunchKernelGGL((k_moe_combine_bwd<KJ, false, false>), dim3((unsigned)g), dim3(kThreads), 0,
                         s, p, tb, share, dy, ys, weight, dys, dw);
  });
  return hipGetLastError();
}

}  // namespace fp8sg
