// gemm_seg.h -- the tiled kernel of the products that gemm.hip does not do:
// rows in segments by expert, and 4-bit operands.
//
//   rows:  C[r][n] = sum_k A[r][k] W_e[n][k]     r in segment e of A's rows
//   depth: C_e[m][n] = sum_{k in segment e} A[m][k] B[n][k]
// each with the operands' scales (tensor, block, MX) and FP32 accumulation.
// Segment e is [offsets[e], offsets[e + 1]), read on the device; without
// offsets there is one segment, all rows.
//
// Design, as gemm.hip: 8 waves a workgroup, an output tile of BM x 256, the
// operands' tiles of one step straight from memory into one of two LDS stages
// (buffer_load ... lds) while the MFMAs work on the other, scales of 512 K by
// the same way.  A step is 128 bytes of a row: 128 K, or 256 K where both
// operands have 4 bits, whose v_mfma takes half the time; a 4-bit operand
// beside an 8-bit one has rows of 64 bytes a step.  What is different:
//   * a workgroup finds its expert itself: every wave scans the segments'
//     tile counts, 64 experts at a time, so the host need not know them;
//   * loads and stores end with the segment, not with the matrix;
//   * BM = 128 (waves 2 x 4 instead of 4 x 2) where segments are short;
//   * depth: a row's stride and the length of its segment are two numbers.
#pragma once

#include "gemm_common.h"
#include "launch.h"

namespace fp8sg {

namespace {

namespace seg {

constexpr int kE2M1 = 4;
constexpr int BN = 256, NT = 512, NW = 8;

struct SegArgs {
  Args g;                  // M: rows of A; C: of expert 0
  const int32_t* offsets;  // or NULL: one segment
  int experts;
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
// `count` tile rows and the tile columns.  `at`: the workgroup's number, dealt
// out in contiguous ranges to the XCDs (XCD) or as it is.
struct Place {
  int e, from, to, count, local;
};
template <int BM, bool XCD>
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
  if constexpr (XCD) {
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
  return RB == 128 ? (row >> 1) & 7 : (row >> 2) & 3;
}
template <int RB>
__device__ __forceinline__ int place(int row, int chunk) {
  return row * RB + ((chunk ^ turn<RB>(row)) << 4);
}

// Moves an operand's ROWS x RB-byte tile of a step into LDS, 1 KB a wave and
// load, lane l to byte 16 l of it.  `stride`: bytes from row to row; `depth`:
// bytes of a row that belong to the product, chunks past it read as zeros, as
// do rows past `rows`.
template <int ROWS, int RB>
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
    const uint4 lo = *reinterpret_cast<const uint4*>(s + place<RB>(r, g));
    const uint4 hi = *reinterpret_cast<const uint4*>(s + place<RB>(r, g + 4));
    o[0] = lo.x; o[1] = lo.y; o[2] = lo.z; o[3] = lo.w;
    o[4] = hi.x; o[5] = hi.y; o[6] = hi.z; o[7] = hi.w;
  }
  return o;
}

// MODE: tensor, block (BRB: rows of B a scale) or MX.  DIRECT (MX rows of a
// length that is no multiple of 128, whose scale bytes are not aligned
// dwords): every lane loads its scale bytes from memory, one step ahead.
template <int MODE, int FA, int FB, int BRB, int BM, bool DEPTH, bool DIRECT>
__global__ __launch_bounds__(NT) __attribute__((amdgpu_waves_per_eu(2, 2)))
void k_gemm_seg(SegArgs p) {
  static_assert(BM == 256 || BM == 128, "tile rows");
  static_assert(!DIRECT || (MODE == kMX && !DEPTH), "scale bytes from memory");
  constexpr bool STAGED = MODE != kTensor && !DIRECT;
  constexpr int KS = FA == kE2M1 && FB == kE2M1 ? 256 : 128, SUB = KS / 128;
  constexpr int RA = FA == kE2M1 ? KS / 2 : KS, RB = FB == kE2M1 ? KS / 2 : KS;
  constexpr int WAVES_M = BM / 64, WN = BN * WAVES_M / NW;
  constexpr int NF = 4, NJ = WN / 16;
  constexpr int A_BYTES = BM * RA, B_BYTES = BN * RB, STAGE = A_BYTES + B_BYTES;
  static_assert(2 * STAGE >= 128 * 512, "half an output tile is staged in LDS");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2][STAGE];
  __shared__ __attribute__((aligned(16))) uint32_t lS[STAGED ? 2 : 1][STAGED ? (BM + BN) * 4 : 4];
  __shared__ uint32_t red[NT / 64];
  Place at;
  int tm, tn;
  if constexpr (DEPTH) {
    // every expert's tiles spread over the XCDs by themselves: the experts'
    // depths differ
    const int T = p.g.tiles_m * p.g.tiles_n, grid = (T + 7) / 8 * 8;
    at.e = blockIdx.x / grid;
    const int b = blockIdx.x - at.e * grid, t = (b & 7) * (grid / 8) + (b >> 3);
    if (t >= T) return;
    walk(t, p.g.tiles_m, p.g.tiles_n, tm, tn);
    const int rows = (int)p.g.K;             // A's and B's row length: all segments
    constexpr int unit = MODE == kTensor ? 16 : 128;
    at.from = min(max(p.offsets[at.e], 0), rows) / unit * unit;
    at.to = max(min(p.offsets[at.e + 1], rows) / unit * unit, at.from);
  } else {
    if (!find<BM, true>(p, p.g.tiles_n, blockIdx.x, at)) return;
    walk(at.local, at.count, p.g.tiles_n, tm, tn);
  }
  const int64_t n0 = (int64_t)tn * BN;
  // the tile's first row of A and of C, and C's rows that this tile may write
  const int64_t m0 = (DEPTH ? 0 : at.from) + (int64_t)tm * BM;
  const int64_t m_end = DEPTH ? p.g.M : at.to;
  const int64_t depth = DEPTH ? at.to - at.from : p.g.K;       // K of the product
  const int lane = threadIdx.x & 63, w = wave_id();
  const int wm = w % WAVES_M, wn = w / WAVES_M;
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
  Loader<BM, RA> la;
  Loader<BN, RB> lb;
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
      if (w < BM / 64)
        ls.init(sa, (int)min(m_end - m0, (int64_t)BM), 1, row_bytes, bytes, w);
      else
        ls.init(sb, (int)min(p.g.N - n0, (int64_t)BN), BRB, row_bytes, bytes, w - BM / 64);
    }
  }
  constexpr int CHUNK = 512 / KS;                              // steps of 512 K
  auto issue = [&](int stage, int kt) {
    la.load(lds[stage], kt);
    lb.load(lds[stage] + A_BYTES, kt);
    if constexpr (STAGED)
      if (kt % CHUNK == 0 && w < (BM + BN) / 64)
        ls.load(lds_addr(&lS[(kt / CHUNK) & 1][w * 256]), kt / CHUNK);
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
        const int r = wm * 64 + f * 16 + lr;
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
    issue(0, 0);
    if constexpr (DIRECT) fetch(now, 0);
  }
  wait_vm<0>();
  __syncthreads();

  for (int kt = 0; kt < nk; ++kt) {
    const int cur = kt & 1;
    const uint8_t* As = lds[cur];
    const uint8_t* Bs = lds[cur] + A_BYTES;
    const uint32_t* S = lS[STAGED ? (kt / CHUNK) & 1 : 0];
    const uint8_t* S8 = reinterpret_cast<const uint8_t*>(S);
    const float* Sf = reinterpret_cast<const float*>(S);
#pragma unroll
    for (int h = 0; h < SUB; ++h) {
      // past the end of K the data are zeros, but the scale bytes may be NaN
      if (SUB > 1 && h > 0 && (int64_t)kt * KS + h * 128 >= depth) break;
      const int sw = (kt % CHUNK) * SUB + h;
      v8i af[NF], bf[2];
#pragma unroll
      for (int f = 0; f < NF; ++f) af[f] = fragment<FA, RA>(As, wm * 64 + f * 16, h);
      bf[0] = fragment<FB, RB>(Bs, wn * WN, h);
      float sa_f[NF];
      int ea[NF], eb[2];
      const int brow = BM + wn * WN;          // scale row of this wave's first column
      if constexpr (MODE == kBlock) {
#pragma unroll
        for (int f = 0; f < NF; ++f) sa_f[f] = Sf[(wm * 64 + f * 16 + lr) * 4 + sw];
        if constexpr (BRB == 128) {
          const float sb_u = Sf[brow * 4 + sw];
#pragma unroll
          for (int f = 0; f < NF; ++f) sa_f[f] *= sb_u;
        }
      } else if constexpr (MODE == kMX && STAGED) {
#pragma unroll
        for (int f = 0; f < NF; ++f) ea[f] = S8[((wm * 64 + f * 16 + lr) * 4 + sw) * 4 + g];
        eb[0] = S8[((brow + lr) * 4 + sw) * 4 + g];
      }
      if (h == 0 && kt + 1 < nk) {
        issue(cur ^ 1, kt + 1);
        if constexpr (DIRECT) fetch(next, kt + 1);
      }
      __builtin_amdgcn_sched_barrier(0);
      v4f P[2][NF];
      const auto promote = [&](int j) {       // acc += scales * P of column j
        if constexpr (MODE == kBlock) {
          float b[4] = {1.f, 1.f, 1.f, 1.f};
          if constexpr (BRB == 1) {
#pragma unroll
            for (int r = 0; r < 4; ++r) b[r] = Sf[(brow + j * 16 + 4 * g + r) * 4 + sw];
          }
#pragma unroll
          for (int f = 0; f < NF; ++f)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              acc[f][j][r] += (BRB == 1 ? sa_f[f] * b[r] : sa_f[f]) * P[j & 1][f][r];
        }
      };
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        if (j + 1 < NJ) {
          bf[(j + 1) & 1] = fragment<FB, RB>(Bs, wn * WN + (j + 1) * 16, h);
          if constexpr (MODE == kMX && STAGED)
            eb[(j + 1) & 1] = S8[((brow + (j + 1) * 16 + lr) * 4 + sw) * 4 + g];
        }
        if constexpr (MODE == kTensor) {
#pragma unroll
          for (int f = 0; f < NF; ++f) acc[f][j] = mfma<FB, FA>(bf[j & 1], af[f], acc[f][j]);
        } else if constexpr (MODE == kMX) {
#pragma unroll
          for (int f = 0; f < NF; ++f)
            acc[f][j] = mfma_mx<FB, FA>(bf[j & 1], af[f], acc[f][j],
                                        STAGED ? eb[j & 1] : now.b[h][j],
                                        STAGED ? ea[f] : now.a[h][f]);
        } else {
#pragma unroll
          for (int f = 0; f < NF; ++f)
            P[j & 1][f] = mfma<FB, FA>(bf[j & 1], af[f], v4f{0.f, 0.f, 0.f, 0.f});
          // column j's MFMAs stay ahead of column j - 1's scaling
          __builtin_amdgcn_sched_barrier(0);
          if (j > 0) promote(j - 1);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (MODE == kBlock) promote(NJ - 1);
    }
    if constexpr (DIRECT) now = next;
    wait_vm<0>();
    __syncthreads();
  }

  // Epilogue, as gemm.hip's.
  const float qs = out.Cq != nullptr ? *out.q_scale : 1.0f;
  uint32_t mx = 0;
  float s = 1.0f;
  if constexpr (MODE == kTensor)
    s = static_cast<const float*>(p.g.sa)[0] * static_cast<const float*>(p.g.sb)[DEPTH ? 0 : at.e];
  if (out.out == 0 && out.Cq == nullptr && out.part == nullptr && (out.N & 7) == 0) {
    // 128 rows of 512 bytes at a time through LDS, 16-byte chunks XOR-swizzled
    // by row, so that global stores cover whole rows
    uint8_t* stage = &lds[0][0];
#pragma unroll
    for (int part = 0; part < BM / 128; ++part) {
      if (part > 0) __syncthreads();
      if (wm / 2 == part) {
#pragma unroll
        for (int f = 0; f < NF; ++f)
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            const v4f a = acc[f][j];
            const int r = (wm & 1) * 64 + f * 16 + lr, c = wn * WN + j * 16 + 4 * g;
            *reinterpret_cast<uint2*>(stage + r * 512 + (((c >> 3) ^ (r & 31)) << 4) +
                                      ((c >> 2) & 1) * 8) =
                make_uint2(pack_bf16x2(a[0] * s, a[1] * s), pack_bf16x2(a[2] * s, a[3] * s));
          }
      }
      __syncthreads();
      const int t = threadIdx.x, ch = t & 31;
#pragma unroll 4
      for (int k = 0; k < 8; ++k) {
        const int r = k * 16 + (t >> 5);
        const int64_t m = m0 + part * 128 + r, n = n0 + ch * 8;
        if (m < m_end && n < out.N)
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out.C) + m * out.N + n) =
              *reinterpret_cast<const uint4*>(stage + r * 512 + ((ch ^ (r & 31)) << 4));
      }
    }
    return;
  }
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    const int64_t m = m0 + wm * 64 + f * 16 + lr;
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

// Workgroups for tiles of bm x bn; with offsets at most one tile row more an
// expert than the rows alone would need.  A multiple of 8, so that every XCD
// gets the same count.
inline int64_t tiles_at_most(const SegProblem& q, int bm, int bn, bool depth) {
  const int64_t tn = (q.N + bn - 1) / bn, tm = (q.M + bm - 1) / bm;
  if (depth) return (tm * tn + 7) / 8 * 8 * q.experts;
  const int64_t more = q.offsets ? (q.M < q.experts ? q.M : q.experts) : 0;
  return ((q.offsets ? q.M / bm + more : tm) * tn + 7) / 8 * 8;
}

inline SegArgs seg_args(const SegProblem& q, int bm) {
  SegArgs a;
  a.g.A = q.A; a.g.B = q.B; a.g.sa = q.sa; a.g.sb = q.sb; a.g.C = q.C; a.g.out = q.out;
  a.g.Cq = q.Cq; a.g.q_scale = q.q_scale; a.g.q_fmt = q.q_fmt; a.g.part = q.part;
  a.g.M = q.M; a.g.N = q.N; a.g.K = q.K;
  a.g.tiles_m = (int)((q.M + bm - 1) / bm);
  a.g.tiles_n = (int)((q.N + BN - 1) / BN);
  a.offsets = q.offsets;
  a.experts = q.experts;
  return a;
}

template <int MODE, int FA, int FB, int BRB, int BM, bool DEPTH, bool DIRECT>
hipError_t run(const SegProblem& q, hipStream_t s) {
  const SegArgs a = seg_args(q, BM);
  const int64_t T = tiles_at_most(q, BM, BN, DEPTH);
  if (T > kMaxGrid) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((k_gemm_seg<MODE, FA, FB, BRB, BM, DEPTH, DIRECT>), dim3((unsigned)T),
                     dim3(NT), 0, s, a);
  return hipGetLastError();
}

}  // namespace seg

}  // namespace
}  // namespace fp8sg
