// gemm_seg.h -- the tiled kernel of the products that gemm.hip does not do:
// rows in segments by expert, and 4-bit operands.
//
//   rows:  C[r][n] = sum_k A[r][k] W_e[n][k]     r in segment e of A's rows
//   depth: C_e[m][n] = sum_{k in segment e} A[m][k] B[n][k]
// each with the operands' scales (tensor, block, MX) and FP32 accumulation.
// Segment e is [offsets[e], offsets[e + 1]), read on the device; without
// offsets there is one segment, all rows.
//
// Design, as gemm.hip: an output tile a workgroup, the operands' tiles of one
// step straight from memory into one of the LDS stages (buffer_load ... lds)
// while the MFMAs work on another, scales of 512 K by the same way.  A step is
// 128 bytes of a row: 128 K, or 256 K where both operands have 4 bits, whose
// v_mfma takes half the time; a 4-bit operand beside an 8-bit one has rows of
// 64 bytes a step.  What is different:
//   * a workgroup finds its expert itself: every wave scans the segments'
//     tile counts, 64 experts at a time, so the host need not know them;
//   * loads and stores end with the segment, not with the matrix;
//   * smaller tiles where segments are short;
//   * depth: a row's stride and the length of its segment are two numbers.
//
// What bounds it, and measured times:
//   long segments: the matrix cores, whose clock falls to 1.9 GHz under such
//     products.  8192 tokens to 2 of 8 experts, 4096 -> 11008, blockwise
//     scales 760 to 779 us (1944 TFLOP/s), its weight gradient under MX 765 us
//     (1930); 4096 x 49152 x 12288 with both operands in 4 bits 1224 to 1258 us
//     (4040), where LDS reads and the operands' loads bound it too (the MFMAs
//     are busy 46 to 48 % of the time, LDS 37 %; without the loads of operands
//     it would take 22 % less, without those of scales 5 %, without B's LDS
//     reads 7 %).
//   short segments: the weights' bytes.  16 tokens to 2 of 8 experts, 4096 ->
//     11008, 4-bit weights 41.5 us (4.6 TB/s); 1000 tokens to 6 of 64 experts,
//     2000 -> 1408, 57.7 us (3.6 TB/s; 480 tokens, which have one tile row an
//     expert, 48 us and 4.1: two tile rows ask for the same weights at the
//     same time, so that fewer bytes are on their way).
//   one row: latency; 11008 x 4096 4-bit weights 7.9 us a call, 172 tiles.
#pragma once

#include "gemm_common.h"
#include "launch.h"

namespace fp8sg {

namespace {

namespace seg {

constexpr int kE2M1 = 4;

struct SegArgs {
  Args g;                  // M: rows of A; C: of expert 0
  const int32_t* offsets;  // or NULL: one segment
  int experts;
  bool stream;             // C is written past the caches
};

// Tile rows of segment e, and where it lies; never outside [0, rows).
__device__ __forceinline__ int tiles_of(const SegArgs& p, int e, int bm, int& from, int& to) {
  from = to = 0;
  if (e >= p.experts) return 0;
  const int rows = (int)p.g.M;
  from = min(max(p.offsets[e], 0), rows);
  to = min(max(p.offsets[e + 1], from), rows);
  return (int)(((int64_t)(to - from) + bm - 1) / bm);
}
__device__ __forceinline__ int wave_scan(int v) {
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int o = __shfl_up(v, off, 64);
    if ((int)(threadIdx.x & 63) >= off) v += o;
  }
  return v;
}
__device__ __forceinline__ int lane_value(int v, int lane) {
  return __builtin_amdgcn_readlane(v, lane);
}

// One output tile: expert, its rows [from, to) and the tile's place among
// `count` tile rows and the tile columns.  `at`: the workgroup's number; the
// XCDs, which take workgroups in turn, get contiguous ranges of the tiles.
struct Place {
  int e, from, to, count, local;
};
template <int BM>
__device__ __forceinline__ bool find(const SegArgs& p, int tiles_n, int at, Place& w) {
  const int lane = threadIdx.x & 63;
  int from, to, n = 0, upto = 0, total = 0;
  if (p.offsets == nullptr) {
    total = p.g.tiles_m;
  } else {
    for (int c = 0; c < p.experts; c += 64) {
      n = tiles_of(p, c + lane, BM, from, to);
      upto = wave_scan(n);
      total += lane_value(upto, 63);
    }
  }
  const int T = total * tiles_n;
  int t = at;
  {                                            // its XCD's range
    const int per = (T + 7) / 8;
    if ((at >> 3) >= per) return false;
    t = (at & 7) * per + (at >> 3);
  }
  if (t >= T) return false;
  if (p.offsets == nullptr) {
    w.e = 0;
    w.from = 0;
    w.to = (int)p.g.M;
    w.count = total;
    w.local = t;
    return true;
  }
  int before = 0;
  for (int c = 0; c < p.experts; c += 64) {
    if (p.experts > 64) {
      n = tiles_of(p, c + lane, BM, from, to);
      upto = wave_scan(n);
    }
    const uint64_t hit = __ballot(t < (before + upto) * tiles_n);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      w.e = c + l;
      w.from = lane_value(from, l);
      w.to = lane_value(to, l);
      w.count = lane_value(n, l);
      w.local = t - (before + lane_value(upto, l) - w.count) * tiles_n;
      return true;
    }
    before += lane_value(upto, 63);
  }
  return false;
}
// A segment's tiles in groups of 8 tile rows, so that neighbours share A rows
// and B rows in an XCD's L2.
__device__ __forceinline__ void walk(int t, int tiles_m, int tiles_n, int& tm, int& tn) {
  constexpr int G = 8;
  const int group = t / (G * tiles_n);
  const int first = group * G;
  const int size = min(tiles_m - first, G);
  const int in = t - group * G * tiles_n;
  tm = first + in % size;
  tn = in / size;
}

// LDS rows of RB bytes a step; 16-byte chunk c of row r lies at slot
// c ^ turn(r), so that the 16 rows of a fragment read fall into all banks.
template <int RB>
__device__ __forceinline__ int turn(int row) {
  return RB == 256 ? row & 15 : RB == 128 ? (row >> 1) & 7 : (row >> 2) & 3;
}
template <int RB>
__device__ __forceinline__ int place(int row, int chunk) {
  return row * RB + ((chunk ^ turn<RB>(row)) << 4);
}

// Moves an operand's ROWS x RB-byte tile of a step into LDS, 1 KB a wave and
// load, lane l to byte 16 l of it.  `stride`: bytes from row to row; `depth`:
// bytes of a row that belong to the product, chunks past it read as zeros, as
// do rows past `rows`.
template <int ROWS, int RB, int NW>
struct Loader {
  static constexpr int L = ROWS * RB / (1024 * NW);
  static constexpr int R = 1024 / RB;           // rows of a load
  v4i rsrc;
  uint32_t records;
  int depth;
  int voff[L], chunk[L];
  int w;
  __device__ __forceinline__ void init(const uint8_t* base, int64_t rows, int64_t stride,
                                       int64_t depth_, int wave) {
    w = wave;
    depth = (int)depth_;
    const int n = (int)(rows < ROWS ? rows : ROWS);
    records = n > 0 && depth_ > 0 ? (uint32_t)((int64_t)(n - 1) * stride + depth_) : 0u;
    records = __builtin_amdgcn_readfirstlane(records);
    rsrc = make_rsrc(base, records);
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < L; ++i) {
      const int row = (w * L + i) * R + lane / (RB / 16);
      chunk[i] = ((lane & (RB / 16 - 1)) ^ turn<RB>(row)) * 16;
      voff[i] = row < n ? (int)(row * stride) + chunk[i] : -1;
    }
  }
  __device__ __forceinline__ void load(const uint8_t* tile, int kt) const {
    const int k0 = kt * RB;
#pragma unroll
    for (int i = 0; i < L; ++i)
      dma16(rsrc, lds_addr(tile) + (uint32_t)((w * L + i) * 1024),
            voff[i] >= 0 && k0 + chunk[i] < depth ? voff[i] + k0 : (int)records);
  }
};

// Four dwords of scales a row and 512 K (FP32 of 128-K blocks, or the E8M0
// bytes of 16 blocks), row r's at LDS word 4 r: wave `part` moves 64 rows.
struct Scales {
  v4i rsrc;
  int voff;
  uint32_t records;
  __device__ __forceinline__ void init(const uint8_t* base, int rows, int br, int64_t stride,
                                       int64_t bytes, int part) {
    const int groups = (rows + br - 1) / br;
    records = groups > 0 && bytes > 0 ? (uint32_t)((groups - 1) * stride + bytes) : 0u;
    records = __builtin_amdgcn_readfirstlane(records);
    rsrc = make_rsrc(base, records);
    const int r = part * 64 + (int)(threadIdx.x & 63);
    voff = r < rows ? (int)((r / br) * stride) : -1;
  }
  __device__ __forceinline__ void load(uint32_t lds, int chunk) const {
    dma16(rsrc, lds, voff >= 0 ? voff + chunk * 16 : (int)records);
  }
};

// 16 rows' MFMA operand of sub-step h, in the order of K that the instruction
// pairs with the other operand's: an 8-bit lane holds K 16 g .. 16 g + 15 and
// 64 + 16 g .. (g = lane / 16), a 4-bit lane K 32 g .. 32 g + 31.
template <int FMT, int RB>
__device__ __forceinline__ v8i fragment(const uint8_t* __restrict__ s, int row0, int h) {
  const int l = threadIdx.x & 63;
  const int r = row0 + (l & 15), g = l >> 4;
  v8i o = {};
  if constexpr (FMT == kE2M1) {
    const uint4 v = *reinterpret_cast<const uint4*>(s + place<RB>(r, 4 * h + g));
    o[0] = v.x; o[1] = v.y; o[2] = v.z; o[3] = v.w;
  } else {
    const uint4 lo = *reinterpret_cast<const uint4*>(s + place<RB>(r, 8 * h + g));
    const uint4 hi = *reinterpret_cast<const uint4*>(s + place<RB>(r, 8 * h + g + 4));
    o[0] = lo.x; o[1] = lo.y; o[2] = lo.z; o[3] = lo.w;
    o[4] = hi.x; o[5] = hi.y; o[6] = hi.z; o[7] = hi.w;
  }
  return o;
}

// 16 bytes of outputs.  `stream`: so many are written in all (kStreamBytes) that a
// later reader would not find them in a cache; past the caches, they leave
// the operands there.  8192 tokens to 2 of 8 experts, 4096 -> 11008: the
// weight gradient 813 -> 784 us; 1000 tokens to 6 of 64 experts, 2000 x 1408
// each: 135 -> 114; dense 8192 x 16384 x 1024 with 4-bit operands 154 -> 127.
template <class V>
__device__ __forceinline__ void store16(void* to, V v, bool stream) {
  static_assert(sizeof(V) == 16, "a chunk");
  V* at = static_cast<V*>(to);
  if (stream) {
    asm volatile("");      // keeps the branch's two stores from becoming one
    __builtin_nontemporal_store(v, at);
    asm volatile("");
  } else {
    *at = v;
  }
}

// The output tile, its waves (each a part of the tile), the LDS stages, and the
// bytes of a row in a step.
template <int BM_, int BN_, int WAVES_M_, int WAVES_N_, int STAGES_, int ROW_ = 128>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, WAVES_M = WAVES_M_, WAVES_N = WAVES_N_;
  static constexpr int STAGES = STAGES_, ROW = ROW_, NW = WAVES_M * WAVES_N, NT = 64 * NW;
  static constexpr int WM = BM / WAVES_M, WN = BN / WAVES_N;
};

// MODE: tensor, block (BRB: rows of B a scale) or MX.  DIRECT (MX rows of a
// length that is no multiple of 128, whose scale bytes are not aligned
// dwords): every lane loads its scale bytes from memory, one step ahead.  Loads
// return in order, so the wait for a step's bytes is one for all operands that
// were asked for before them: the tiles of three or four stages have one step
// on its way, as those of two.  K = 4096 against 4064 and 4160 (us): 16 tokens
// to 2 of 8 experts with 4-bit weights 45.6, 75.0, 74.4; 512 tokens with 8-bit
// ones 129, 253, 230; 8192 tokens 745, 1284, 1233; one row through 4-bit weights
// 8.4, 14.5, 14.8; 4096 rows of 4 bits 122, 228, 225 (11008 columns all).
template <int MODE, int FA, int FB, int BRB, class T, bool DEPTH, bool DIRECT>
__global__ __launch_bounds__(T::NT) __attribute__((amdgpu_waves_per_eu(2)))
void k_gemm_seg(SegArgs p) {
  static_assert(!DIRECT || (MODE == kMX && !DEPTH), "scale bytes from memory");
  constexpr int BM = T::BM, BN = T::BN, NW = T::NW, NT = T::NT, STAGES = T::STAGES;
  constexpr bool STAGED = MODE != kTensor && !DIRECT;
  constexpr int KS = FA == kE2M1 && FB == kE2M1 ? 2 * T::ROW : T::ROW, SUB = KS / 128;
  constexpr int RA = FA == kE2M1 ? KS / 2 : KS, RB = FB == kE2M1 ? KS / 2 : KS;
  constexpr int WM = T::WM, WN = T::WN, NF = WM / 16, NJ = WN / 16;
  constexpr int A_BYTES = BM * RA, B_BYTES = BN * RB, STAGE = A_BYTES + B_BYTES;
  constexpr int CHUNK = 512 / KS;              // steps of 512 K of scales
  // columns that a B fragment is read before its products
  constexpr int AHEAD = 1;
  // chunks that the steps in flight and the present one can be of
  constexpr int CHUNKS = (STAGES - 2 + CHUNK) / CHUNK + 1;
  // scale rows, A's first, 64 a wave's load
  constexpr int AS = (BM + 63) / 64, BS = (BN + 63) / 64, SW = AS + BS;
  static_assert(SW <= NW, "64 rows of scales a wave");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[STAGES][STAGE];
  __shared__ __attribute__((aligned(16))) uint32_t lS[STAGED ? CHUNKS : 1][STAGED ? SW * 256 : 4];
  __shared__ uint32_t red[NW];
  Place at;
  int tm, tn;
  if constexpr (DEPTH) {
    // every expert's tiles spread over the XCDs by themselves: the experts'
    // depths differ
    const int tiles = p.g.tiles_m * p.g.tiles_n, grid = (tiles + 7) / 8 * 8;
    at.e = blockIdx.x / grid;
    const int b = blockIdx.x - at.e * grid, t = (b & 7) * (grid / 8) + (b >> 3);
    if (t >= tiles) return;
    walk(t, p.g.tiles_m, p.g.tiles_n, tm, tn);
    const int rows = (int)p.g.K;             // A's and B's row length: all segments
    constexpr int unit = MODE == kTensor ? 16 : 128;
    at.from = min(max(p.offsets[at.e], 0), rows) / unit * unit;
    at.to = max(min(p.offsets[at.e + 1], rows) / unit * unit, at.from);
  } else {
    if (!find<BM>(p, p.g.tiles_n, blockIdx.x, at)) return;
    walk(at.local, at.count, p.g.tiles_n, tm, tn);
  }
  const int64_t n0 = (int64_t)tn * BN;
  // the tile's first row of A and of C, and C's rows that this tile may write
  const int64_t m0 = (DEPTH ? 0 : at.from) + (int64_t)tm * BM;
  const int64_t m_end = DEPTH ? p.g.M : at.to;
  const int64_t depth = DEPTH ? at.to - at.from : p.g.K;       // K of the product
  const int lane = threadIdx.x & 63, w = wave_id();
  const int wm = w / T::WAVES_N, wn = w % T::WAVES_N;
  const int g = lane >> 4, lr = lane & 15;
  const int nk = (int)((depth + KS - 1) / KS);
  Args out = p.g;
  if constexpr (DEPTH) {
    const int64_t skip = at.e * p.g.M * p.g.N;
    out.C = static_cast<uint8_t*>(p.g.C) + skip * (p.g.out == 0 ? 2 : 4);
  }

  v4f acc[NF][NJ];
#pragma unroll
  for (int f = 0; f < NF; ++f)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[f][j] = v4f{0.f, 0.f, 0.f, 0.f};

  constexpr int DA = FA == kE2M1 ? 2 : 1, DB = FB == kE2M1 ? 2 : 1;   // elements a byte
  const int64_t lda = p.g.K / DA, ldb = p.g.K / DB;
  Loader<BM, RA, NW> la;
  Loader<BN, RB, NW> lb;
  la.init(p.g.A + m0 * lda + (DEPTH ? at.from / DA : 0), m_end - m0, lda, depth / DA, w);
  lb.init(p.g.B + (DEPTH ? n0 * ldb + at.from / DB : (at.e * p.g.N + n0) * ldb), p.g.N - n0, ldb,
          depth / DB, w);
  // scales: 64 rows a wave, A's rows first
  constexpr int PER = MODE == kBlock ? 128 : 32;               // K of a scale
  constexpr int SB = MODE == kBlock ? 4 : 1;                   // its bytes
  Scales ls;
  const uint8_t* sa = static_cast<const uint8_t*>(p.g.sa);
  const uint8_t* sb = static_cast<const uint8_t*>(p.g.sb);
  if constexpr (MODE != kTensor) {
    const int64_t row_bytes = p.g.K / PER * SB, skip = DEPTH ? at.from / PER * SB : 0;
    sa += m0 * row_bytes + skip;
    sb += (DEPTH ? n0 : (at.e * p.g.N + n0) / BRB) * row_bytes + skip;
    if constexpr (STAGED) {
      const int64_t bytes = (depth + PER - 1) / PER * SB;
      if (w < AS)
        ls.init(sa, (int)min(m_end - m0, (int64_t)BM), 1, row_bytes, bytes, w);
      else
        ls.init(sb, (int)min(p.g.N - n0, (int64_t)BN), BRB, row_bytes, bytes, w - AS);
    }
  }
  // The loads of step kt, as many in every step where more than one is in
  // flight (a step past the end reads nothing); scales come in addition, which
  // makes the wait for a step a little longer than it need be.
  constexpr int LOADS = Loader<BM, RA, NW>::L + Loader<BN, RB, NW>::L;
  int into = 0;                                // the stage of the next step to load
  auto issue = [&](int kt) {
    if constexpr (STAGED) {
      if (kt % CHUNK == 0 && w < SW)
        ls.load(lds_addr(&lS[(kt / CHUNK) % CHUNKS][w * 256]), kt / CHUNK);
    }
    la.load(lds[into], kt);
    lb.load(lds[into] + A_BYTES, kt);
    into = into + 1 == STAGES ? 0 : into + 1;
  };
  // DIRECT: this lane's scale bytes of step kt, 1 where there is no block
  struct Bytes {
    int a[SUB][NF], b[SUB][NJ];
  };
  auto fetch = [&](Bytes& s, int kt) {
    const int64_t row = p.g.K / 32;
#pragma unroll
    for (int h = 0; h < SUB; ++h) {
      const int64_t blk = ((int64_t)kt * SUB + h) * 4 + g;
      const bool in = blk < row;
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        const int r = wm * WM + f * 16 + lr;
        s.a[h][f] = in && m0 + r < m_end ? sa[r * row + blk] : 127;
      }
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int r = wn * WN + j * 16 + lr;
        s.b[h][j] = in && n0 + r < p.g.N ? sb[r * row + blk] : 127;
      }
    }
  };
  Bytes now, next;

  if (nk > 0) {
    if constexpr (DIRECT) fetch(now, 0);
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i)
      if (STAGES > 2 || i < nk) issue(i);
  }

  // a wave whose part of the tile is outside the segment or the columns moves
  // data only (waves share their SIMD with one of other rows)
  const bool idle = m0 + wm * WM >= m_end || n0 + wn * WN >= p.g.N;
  int cur = 0;
  for (int kt = 0; kt < nk; ++kt) {
    // step kt has landed, for every wave, and the stage before it is free
    wait_vm<LOADS * (STAGES - 2)>();
    __syncthreads();
    const uint8_t* As = lds[cur];
    const uint8_t* Bs = lds[cur] + A_BYTES;
    cur = cur + 1 == STAGES ? 0 : cur + 1;
    const uint32_t* S = lS[STAGED ? (kt / CHUNK) % CHUNKS : 0];
    const uint8_t* S8 = reinterpret_cast<const uint8_t*>(S);
    const float* Sf = reinterpret_cast<const float*>(S);
    const int brow = AS * 64 + wn * WN;         // scale row of this wave's first column
    // The step's columns of fragments, c = h NJ + j: column c's B fragment is
    // read AHEAD columns before its products, the A fragments of sub-step h
    // among the columns of the sub-step before.
    v8i af[SUB > 1 ? 2 : 1][NF], bf[AHEAD + 1];
    int ea[SUB > 1 ? 2 : 1][NF], eb[AHEAD + 1];
    float sa_f[NF];
    const auto read_a = [&](int h, int f) {
      af[h & (SUB > 1)][f] = fragment<FA, RA>(As, wm * WM + f * 16, h);
      if constexpr (MODE == kMX && STAGED)
        ea[h & (SUB > 1)][f] = S8[((wm * WM + f * 16 + lr) * 4 + (kt % CHUNK) * SUB + h) * 4 + g];
    };
    const auto read_b = [&](int c) {
      const int h = c / NJ, j = c % NJ;
      bf[c % (AHEAD + 1)] = fragment<FB, RB>(Bs, wn * WN + j * 16, h);
      if constexpr (MODE == kMX && STAGED)
        eb[c % (AHEAD + 1)] = S8[((brow + j * 16 + lr) * 4 + (kt % CHUNK) * SUB + h) * 4 + g];
    };
    if (!idle) {
#pragma unroll
      for (int f = 0; f < NF; ++f) read_a(0, f);
#pragma unroll
      for (int c = 0; c < AHEAD; ++c)
        if (c < SUB * NJ) read_b(c);
    }
    if (kt + STAGES - 1 < nk || STAGES > 2) issue(kt + STAGES - 1);
    if constexpr (DIRECT)
      if (kt + 1 < nk) fetch(next, kt + 1);
    if (idle) continue;
    v4f P[2][NF];
    const auto scales_of = [&](int h) {         // block mode: A's, times B's where it is one
      if constexpr (MODE == kBlock) {
        const int sw = (kt % CHUNK) * SUB + h;
#pragma unroll
        for (int f = 0; f < NF; ++f) sa_f[f] = Sf[(wm * WM + f * 16 + lr) * 4 + sw];
        if constexpr (BRB == 128) {
          const float sb_u = Sf[brow * 4 + sw];
#pragma unroll
          for (int f = 0; f < NF; ++f) sa_f[f] *= sb_u;
        }
      }
    };
    const auto promote = [&](int c) {           // acc += scales * P of column c
      if constexpr (MODE == kBlock) {
        const int h = c / NJ, j = c % NJ, sw = (kt % CHUNK) * SUB + h;
        float b[4] = {1.f, 1.f, 1.f, 1.f};
        if constexpr (BRB == 1) {
#pragma unroll
          for (int r = 0; r < 4; ++r) b[r] = Sf[(brow + j * 16 + 4 * g + r) * 4 + sw];
        }
#pragma unroll
        for (int f = 0; f < NF; ++f)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            acc[f][j][r] += (BRB == 1 ? sa_f[f] * b[r] : sa_f[f]) * P[c & 1][f][r];
      }
    };
    scales_of(0);
    bool ended = false;
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int c = 0; c < SUB * NJ; ++c) {
      const int h = c / NJ, j = c % NJ;
      // past the end of K the data are zeros, but the scale bytes may be NaN
      if (h > 0 && j == 0 && (int64_t)kt * KS + h * 128 >= depth) {
        if constexpr (MODE == kBlock) promote(c - 1);
        ended = true;
        break;
      }
      if (c + AHEAD < SUB * NJ) read_b(c + AHEAD);
      if (h + 1 < SUB) {
        if constexpr (NJ > NF) {
          if (j >= NJ - 1 - NF && j < NJ - 1) read_a(h + 1, j - (NJ - 1 - NF));
        } else {
          if (j == 0)
#pragma unroll
            for (int f = 0; f < NF; ++f) read_a(h + 1, f);
        }
      }
      const v8i b = bf[c % (AHEAD + 1)];
      const v8i(&a)[NF] = af[h & (SUB > 1)];
      if constexpr (MODE == kTensor) {
#pragma unroll
        for (int f = 0; f < NF; ++f) acc[f][j] = mfma<FB, FA>(b, a[f], acc[f][j]);
      } else if constexpr (MODE == kMX) {
#pragma unroll
        for (int f = 0; f < NF; ++f)
          acc[f][j] = mfma_mx<FB, FA>(b, a[f], acc[f][j],
                                      STAGED ? eb[c % (AHEAD + 1)] : now.b[h][j],
                                      STAGED ? ea[h & (SUB > 1)][f] : now.a[h][f]);
      } else {
#pragma unroll
        for (int f = 0; f < NF; ++f)
          P[c & 1][f] = mfma<FB, FA>(b, a[f], v4f{0.f, 0.f, 0.f, 0.f});
        // column c's MFMAs stay ahead of column c - 1's scaling
        __builtin_amdgcn_sched_barrier(0);
        if (c > 0) promote(c - 1);
        if (h > 0 && j == 0) scales_of(h);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (MODE == kBlock)
      if (!ended) promote(SUB * NJ - 1);
    if constexpr (DIRECT) now = next;
  }
  wait_vm<0>();
  __syncthreads();

  // Epilogue, as gemm.hip's.
  const float qs = out.Cq != nullptr ? *out.q_scale : 1.0f;
  uint32_t mx = 0;
  float s = 1.0f;
  if constexpr (MODE == kTensor)
    s = static_cast<const float*>(p.g.sa)[0] * static_cast<const float*>(p.g.sb)[DEPTH ? 0 : at.e];
  if (out.out == 0 && out.Cq == nullptr && out.part == nullptr && (out.N & 7) == 0) {
    // up to 128 rows at a time through LDS, 16-byte chunks XOR-swizzled by
    // row, so that global stores cover whole rows
    constexpr int PART = BM < 128 ? BM : 128, CH = BN / 8, ROW = BN * 2, PASS = NT / CH;
    static_assert(PART * ROW <= STAGES * STAGE, "the staged rows");
    uint8_t* stage = &lds[0][0];
#pragma unroll
    for (int part = 0; part < BM / PART; ++part) {
      if (part > 0) __syncthreads();
      if (wm * WM / PART == part) {
#pragma unroll
        for (int f = 0; f < NF; ++f)
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            const v4f a = acc[f][j];
            const int r = (wm * WM) % PART + f * 16 + lr, c = wn * WN + j * 16 + 4 * g;
            *reinterpret_cast<uint2*>(stage + r * ROW + (((c >> 3) ^ (r & (CH - 1))) << 4) +
                                      ((c >> 2) & 1) * 8) =
                make_uint2(pack_bf16x2(a[0] * s, a[1] * s), pack_bf16x2(a[2] * s, a[3] * s));
          }
      }
      __syncthreads();
      const int t = threadIdx.x, ch = t % CH;
#pragma unroll 4
      for (int r = t / CH; r < PART; r += PASS) {
        const int64_t m = m0 + part * PART + r, n = n0 + ch * 8;
        if (m < m_end && n < out.N)
          store16(static_cast<uint16_t*>(out.C) + m * out.N + n,
                  *reinterpret_cast<const v4i*>(stage + r * ROW + ((ch ^ (r & (CH - 1))) << 4)),
                  p.stream);
      }
    }
    return;
  }
  if constexpr (DEPTH) {
    if (out.out != 0 && (out.N & 3) == 0) {
      // FP32, in the same way.  Added to what is there (us; MX), against store4:
      // 8192 tokens to 2 of 8 experts, 4096 x 11008 1147 / 1161; 2048 tokens, 4096
      // x 2048 146 / 163; 1000 tokens to 6 of 64, 2000 x 1408 333 / 386; but 512
      // tokens to 2 of 8, 4096 x 11008 663 / 634.  Stored, past the caches against
      // into them: 886 / 945, 81 / 90, 166 / 199, 331 / 358
      constexpr int PART = BM < 128 ? BM : 128, CH = BN / 4, ROW = BN * 4, PASS = NT / CH;
      static_assert(PART * ROW <= STAGES * STAGE, "the staged rows");
      uint8_t* stage = &lds[0][0];
#pragma unroll
      for (int part = 0; part < BM / PART; ++part) {
        if (part > 0) __syncthreads();
        if (wm * WM / PART == part) {
#pragma unroll
          for (int f = 0; f < NF; ++f)
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
              const int r = (wm * WM) % PART + f * 16 + lr, ch = (wn * WN + j * 16) / 4 + g;
              *reinterpret_cast<v4f*>(stage + r * ROW + ((ch ^ (r & (CH - 1))) << 4)) =
                  acc[f][j] * s;
            }
        }
        __syncthreads();
        const int t = threadIdx.x, ch = t % CH;
        constexpr int U = PART / PASS < 4 ? PART / PASS : 4;   // rows whose old values come together
        float* const to = static_cast<float*>(out.C) + (m0 + part * PART) * out.N + n0 + ch * 4;
        const bool in = n0 + ch * 4 < out.N;
        for (int r0 = t / CH; r0 < PART; r0 += U * PASS) {
          v4f old[U] = {};
          if (out.out == 2) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
              const int r = r0 + u * PASS;
              if (in && m0 + part * PART + r < m_end)
                old[u] = *reinterpret_cast<const v4f*>(to + r * out.N);
            }
          }
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int r = r0 + u * PASS;
            v4f v = *reinterpret_cast<const v4f*>(stage + r * ROW + ((ch ^ (r & (CH - 1))) << 4));
            if (out.out == 2) v = old[u] + v;
            if (in && m0 + part * PART + r < m_end) store16(to + r * out.N, v, p.stream);
          }
        }
      }
      return;
    }
  }
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    const int64_t m = m0 + wm * WM + f * 16 + lr;
    if (m >= m_end) continue;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int64_t n = n0 + wn * WN + j * 16 + 4 * g;
      if (n >= out.N) continue;
      const v4f a = acc[f][j];
      store4(out, m, n, a[0] * s, a[1] * s, a[2] * s, a[3] * s, qs, mx);
    }
  }
  tile_amax<NT>(out, tm, tn, mx, red);
}

// The tiles by TileKind; which one is taken, and the times of its neighbours,
// stand in seg_shape.h.  Large ones read their operands as few times as
// LDS allows.  The smaller ones are for short segments, where loading is all:
// several workgroups a CU, two or three steps on their way beside the one at
// work (16 tokens to 8 experts with 4-bit weights: 96 us with one step on its
// way, 45 with three).  That of 16 rows has steps of 256 bytes a row, twice
// the bytes to a barrier.  64 x 128: three stages of 2 x 2 waves 98.6 us (256
// tokens, 2 of 8 experts, 4096 -> 11008, 8 bits), two stages 113, 2 x 4 waves
// 98.6; 128 x 64 109, 128 x 128 107 to 109.
typedef Tile<256, 256, 4, 2, 2> T256;
typedef Tile<128, 128, 2, 2, 2> T128;
typedef Tile<64, 128, 2, 2, 3> T64x128;
typedef Tile<64, 64, 2, 2, 3> T64;
typedef Tile<32, 64, 1, 4, 4> T32;
typedef Tile<16, 64, 1, 4, 3, 256> T16;

inline SegArgs seg_args(const SegProblem& q, int bm, int bn, bool depth) {
  SegArgs a;
  a.g.A = q.A; a.g.B = q.B; a.g.sa = q.sa; a.g.sb = q.sb; a.g.C = q.C; a.g.out = q.out;
  a.g.Cq = q.Cq; a.g.q_scale = q.q_scale; a.g.q_fmt = q.q_fmt; a.g.part = q.part;
  a.g.M = q.M; a.g.N = q.N; a.g.K = q.K;
  a.g.tiles_m = (int)((q.M + bm - 1) / bm);
  a.g.tiles_n = (int)((q.N + bn - 1) / bn);
  a.offsets = q.offsets;
  a.experts = q.experts;
  a.stream = q.M * q.N * (depth ? q.experts : 1) * (q.out == 0 ? 2 : 4) > kStreamBytes;
  return a;
}

template <int MODE, int FA, int FB, int BRB, class T, bool DEPTH, bool DIRECT>
hipError_t run(const SegProblem& q, hipStream_t s) {
  const SegArgs a = seg_args(q, T::BM, T::BN, DEPTH);
  // every XCD the same count
  const int64_t n = DEPTH ? ((int64_t)a.g.tiles_m * a.g.tiles_n + 7) / 8 * 8 * q.experts
                          : (row_tiles(q.size(), T::BM, T::BN) + 7) / 8 * 8;
  if (n > kMaxGrid) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((k_gemm_seg<MODE, FA, FB, BRB, T, DEPTH, DIRECT>), dim3((unsigned)n),
                     dim3(T::NT), 0, s, a);
  return hipGetLastError();
}
template <int MODE, int FA, int FB, int BRB, bool DIRECT>
hipError_t run_rows(const SegProblem& q, TileKind t, hipStream_t s) {
  switch (t) {
    case kTile256: return run<MODE, FA, FB, BRB, T256, false, DIRECT>(q, s);
    case kTile128: return run<MODE, FA, FB, BRB, T128, false, DIRECT>(q, s);
    case kTile64x128: return run<MODE, FA, FB, BRB, T64x128, false, DIRECT>(q, s);
    case kTile64: return run<MODE, FA, FB, BRB, T64, false, DIRECT>(q, s);
    case kTile32: return run<MODE, FA, FB, BRB, T32, false, DIRECT>(q, s);
    case kTile16: break;
  }
  if constexpr (FB == kE2M1) return run<MODE, FA, FB, BRB, T16, false, DIRECT>(q, s);
  return hipErrorInvalidValue;
}

}  // namespace seg

}  // namespace
}  // namespace fp8sg
