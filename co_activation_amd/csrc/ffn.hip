// The experts' gated feed-forward block over rows grouped by expert, forward
// and backward (the computation between moe_expert_plan's layout and the
// combine of the replies):
//
//   [g | u] = x Win_e^T     Win_e [2F][H]: F gate rows, then F up rows
//   a = act(g) * u          act(g) = g sigmoid(g), or g Phi(g)
//   y = a Wdown_e^T         Wdown_e [H][F]
//
//   da = dy Wdown_e;  dg = da u act'(g);  du = da act(g)
//   dx = [dg | du] Win_e;  dWin_e = [dg | du]^T x;  dWdown_e = dy^T a
//
// Forward: one launch forms gate and up side by side (a wave's 64 columns are
// 32 of each, the same 32) and multiplies them in its registers, so g and u
// are written only for training; a second launch is the down product.
// Backward: the product with Wdown has the activation's derivative as its
// epilogue; [dg | du] lies in the workspace, in the rows' type (bf16 rows:
// one rounding, as for a, which is what the matrix instructions take; all
// sums are fp32).  Then one product each for dx, dWin and dWdown.  Which
// expert a block works for comes from the row counts on the device, so the
// host never waits for the routing: every block cuts the experts' rows into
// tiles from the counts and finds its own.
//
// Measured on MI355X (bf16): 65536 rows over 64 experts of 4096 x 2048, 3.25 ms
// forward (1.01 PFLOP/s), 6.65 backward (0.99); 24594 uneven rows over 128 of
// 2048 x 1000, 0.53 and 1.3 to 1.4 ms; one token's eight experts of 4096 x 2048,
// 74 us (weights at 5.4 TB/s).
#include <initializer_list>

#include "gemm.hpp"

namespace moe {
namespace {

enum Act { kSilu = MOE_ACT_SILU, kGelu = MOE_ACT_GELU };

// Phi(g), and exp(-g^2 / 2) by the way.  The smaller of the two tails is formed
// as such, exp(-a^2 / 2) Q(a) with a = |g|, and Phi is it or its complement: 1 +
// erf(g / sqrt 2) loses a bit with every factor of two by which Phi is below 1,
// all of them at g = -6.  Q(a) = erfcx(a / sqrt 2) / 2 is t = 1 / (1 + 0.35 a)
// times a polynomial in t, fitted here for the least largest relative error over
// 0 <= a <= 15: 3.2e-8, and 3.3e-7 as evaluated in fp32.  The exponential's
// argument is rounded, so the tail is off by about a^2 2^-24 of itself besides,
// as much as a last digit of g is worth.  From a = 15 on it is 0 in fp32, and
// infinities take that value.
__device__ __forceinline__ float normal_cdf(float g, float& density) {
  const float a = fminf(fabsf(g), 15.f);
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.35f, a, 1.f));
  float q = -0.0291634817f;
  q = __builtin_fmaf(q, t, 0.144058883f);
  q = __builtin_fmaf(q, t, -0.255898416f);
  q = __builtin_fmaf(q, t, 0.159389555f);
  q = __builtin_fmaf(q, t, -0.0232619252f);
  q = __builtin_fmaf(q, t, 0.105574153f);
  q = __builtin_fmaf(q, t, 0.119815625f);
  q = __builtin_fmaf(q, t, 0.139864326f);
  q = __builtin_fmaf(q, t, 0.139621258f);
  density = __expf(-0.5f * a * a);
  const float tail = density * (q * t);
  return g < 0.f ? tail : 1.f - tail;
}

// act(g) and its derivative.  The reciprocal is the instruction's (1 ulp): a
// correctly rounded division is ten, on 128 values a lane and tile.
__device__ __forceinline__ void act_both(int act, float g, float& value, float& slope) {
  if (act == kSilu) {
    const float s = __builtin_amdgcn_rcpf(1.f + __expf(-g));
    value = g * s;
    slope = s * (1.f + g * (1.f - s));
  } else {
    float density;
    const float p = normal_cdf(g, density);
    value = g * p;
    slope = __builtin_fmaf(g * 0.39894228f, density, p);
  }
}

__device__ __forceinline__ float act_value(int act, float g) {
  if (act == kSilu) return g * __builtin_amdgcn_rcpf(1.f + __expf(-g));
  float density;
  return g * normal_cdf(g, density);
}

// ---------------------------------------------------------------- row tiles

// Where each expert's rows lie, on the device.
struct ExpertRows {
  const int32_t* first;
  const int32_t* count;
  int32_t* d_err;
  int E, R;
};

struct RowTile {
  int expert, row, rows;  // first row, rows (1..tile rows)
};

// Row tiles the experts' blocks can need at most, for any disjoint counts.
inline int64_t most_tiles(int64_t R, int E, int bm) { return R / bm + (R < E ? R : E); }

__device__ __forceinline__ int rows_of(const ExpertRows& x, int e, int& first) {
  first = x.first[e];
  const int c = x.count[e];
  if (c >= 0 && first >= 0 && first <= x.R && c <= x.R - first) return c;
  report(x.d_err, MOE_DERR_EXPERT_ROWS);
  return 0;
}

// A block's number -> (row tile, column tile) of mt x nt.  Consecutive blocks
// go to the eight XCDs in turn, each with its own L2: an XCD takes a
// contiguous range of tiles, in panels of kPanel row tiles with the rows
// fastest, so that the blocks it runs together share rows and weights.
constexpr int kXcds = 8;
constexpr int kPanel = 4;

__device__ __forceinline__ bool tile_of(int block, int mt, int nt, int& m, int& n) {
  const int total = mt * nt;
  const int per = (total + kXcds - 1) / kXcds;
  const int i = (block % kXcds) * per + block / kXcds;
  if (block / kXcds >= per || i >= total) return false;
  const int panel = i / (kPanel * nt);
  const int rows = min(kPanel, mt - panel * kPanel);
  const int in = i - panel * kPanel * nt;
  n = in / rows;
  m = panel * kPanel + in - n * rows;
  return true;
}

// The block's row tile and column tile: every expert's rows are cut into
// tiles of bm, in expert order, and each block finds its own from the counts
// (256 of them at most: one load a thread and a scan, no dearer than reading
// a list that another launch would have had to make).  All threads call it,
// at least 256 of them; scratch is LDS of at least 32 bytes, free again when
// the call returns.
__device__ __forceinline__ bool find_tile(const ExpertRows& x, int block, int bm, int nt, char* scratch,
                                          RowTile& t, int& n) {
  static_assert(MOE_MAX_E <= 256, "one expert a thread");
  int* s_wave = reinterpret_cast<int*>(scratch);
  RowTile& s_tile = *reinterpret_cast<RowTile*>(scratch + 16);
  int first = 0, c = 0, tiles = 0, incl = 0;
  if (threadIdx.x == 0) s_tile = {0, 0, 0};
  if (threadIdx.x < 256) {
    if (static_cast<int>(threadIdx.x) < x.E) c = rows_of(x, threadIdx.x, first);
    tiles = (c + bm - 1) / bm;
    incl = wave_incl_scan(tiles);
    if (lane_id() == kWave - 1) s_wave[wave_id()] = incl;
  }
  __syncthreads();
  const int w1 = s_wave[0], w2 = w1 + s_wave[1], w3 = w2 + s_wave[2];
  int m;
  if (!tile_of(block, w3 + s_wave[3], nt, m, n)) return false;
  if (threadIdx.x < 256) {
    const int w = wave_id();
    const int base = incl - tiles + (w == 0 ? 0 : w == 1 ? w1 : w == 2 ? w2 : w3);
    if (m >= base && m < base + tiles) {
      const int at = (m - base) * bm;
      s_tile = {static_cast<int>(threadIdx.x), first + at, min(bm, c - at)};
    }
  }
  __syncthreads();
  t.expert = __builtin_amdgcn_readfirstlane(s_tile.expert);
  t.row = __builtin_amdgcn_readfirstlane(s_tile.row);
  t.rows = __builtin_amdgcn_readfirstlane(s_tile.rows);
  __syncthreads();
  return t.rows > 0;  // none: counts whose sum passes 2^31, so not disjoint
}

// The same for a block that takes one tile after another: the row tiles of
// every expert in LDS.  Block b runs on XCD b % 8 and takes every
// (blocks / 8)-th tile of that XCD's range.
struct ExpertTable {
  int first[256], count[256], upto[256];  // upto: row tiles of experts 0 .. e
  int wave[4];
};

// Fills the table (all threads, at least 256); returns the number of row tiles.
__device__ __forceinline__ int fill_table(const ExpertRows& x, int bm, ExpertTable& t) {
  int first = 0, c = 0, incl = 0;
  if (threadIdx.x < 256) {
    if (static_cast<int>(threadIdx.x) < x.E) c = rows_of(x, threadIdx.x, first);
    incl = wave_incl_scan((c + bm - 1) / bm);
    if (lane_id() == kWave - 1) t.wave[wave_id()] = incl;
  }
  __syncthreads();
  if (threadIdx.x < 256) {
    for (int w = 0; w < wave_id(); ++w) incl += t.wave[w];
    t.first[threadIdx.x] = first;
    t.count[threadIdx.x] = c;
    t.upto[threadIdx.x] = incl;
  }
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(t.upto[255]);
}

// The expert of row tile m: the number of experts whose tiles end before it.
__device__ __forceinline__ int expert_of(const ExpertTable& t, int m) {
  int before = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) before += __popcll(ballot(t.upto[j * kWave + lane_id()] <= m));
  return before;
}

// The block's i-th of `total` tiles, by number: those of an XCD lie together.
__device__ __forceinline__ int block_tile(int i, int total, int block, int blocks) {
  const int per = (total + kXcds - 1) / kXcds;
  const int in = block / kXcds + i * (blocks / kXcds);
  const int t = block % kXcds * per + in;
  return in < per && t < total ? t : -1;
}

// Tile `in` of mt x nt, in panels of kPanel row tiles, rows fastest.
__device__ __forceinline__ void panel_tile(int in, int mt, int nt, int& m, int& n) {
  const int panel = in / (kPanel * nt);
  const int rows = min(kPanel, mt - panel * kPanel);
  const int at = in - panel * kPanel * nt;
  n = at / rows;
  m = panel * kPanel + at - n * rows;
}

// The block's i-th tile of a weight gradient, whose tiles take as long as their
// expert has rows: panels of kPanel tile rows are dealt to the XCDs, there and
// back, so that no XCD has all the long ones (kDealt panels or more; fewer
// would not come out even, and lie together instead).  128 uneven experts of
// 2048 x 1000, 192 rows on average: dWin 490 us, with a range of tiles an XCD
// 565; 64 experts of 4096 x 2048, 1024 rows: 2.35 ms and 2.70.
constexpr int kDealt = 8 * kXcds;

__device__ __forceinline__ bool dealt_tile(int i, int mt, int nt, int block, int blocks, int& m, int& n) {
  const int panels = (mt + kPanel - 1) / kPanel;
  if (panels < kDealt) {
    const int at = block_tile(i, mt * nt, block, blocks);
    if (at < 0) return false;
    panel_tile(at, mt, nt, m, n);
    return true;
  }
  const int in = block / kXcds + i * (blocks / kXcds);
  const int turn = in / (kPanel * nt);
  const int xcd = block % kXcds;
  const int panel = turn * kXcds + ((turn & 1) ? kXcds - 1 - xcd : xcd);
  if (panel >= panels) return false;
  const int rows = min(kPanel, mt - panel * kPanel);
  const int at = in - turn * kPanel * nt;
  n = at / rows;
  m = panel * kPanel + at - n * rows;
  return n < nt;  // a short panel is the last
}

// ---------------------------------------------------------------- bf16 tiles

enum Product {
  kUp,       // a (and g, u) = x Win^T
  kDown,     // y = a Wdown^T
  kActGrad,  // [dg | du] from da = dy Wdown
  kGradX     // dx = [dg | du] Win
};

struct RowArgs {
  const char* a;      // rows, k contiguous
  const char* w;      // weights
  int64_t w_stride;   // bytes of one expert's weights
  char* out;          // a, y, [dg | du] or dx
  char* gu;           // kUp: [g | u] out or null; kActGrad: [g | u] in
  ExpertRows rows;
  int K, N;           // N: F, H, F or H
  int n_blocks;       // column tiles (few rows: groups of n_per of them)
  int n_per;
  int act;
};

__device__ __forceinline__ bf16x4 round4(f32x4 v) { return __builtin_convertvector(v, bf16x4); }

// Stores columns of a row through a buffer: rows and columns outside the tile
// have offsets outside it, so no branch splits the stores.
__device__ __forceinline__ void store4(__amdgpu_buffer_rsrc_t r, int off, f32x4 v) {
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, round4(v)), r, off, 0, 0);
}

__device__ __forceinline__ void store8(__amdgpu_buffer_rsrc_t r, int off, f32x4 lo, f32x4 hi) {
  const bf16x8 v = __builtin_shufflevector(round4(lo), round4(hi), 0, 1, 2, 3, 4, 5, 6, 7);
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), r, off, 0, 0);
}

__device__ __forceinline__ void load8(__amdgpu_buffer_rsrc_t r, int off, f32x4& lo, f32x4& hi) {
  const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0);
  lo = f32x4{bf16_lo(v[0]), bf16_hi(v[0]), bf16_lo(v[1]), bf16_hi(v[1])};
  hi = f32x4{bf16_lo(v[2]), bf16_hi(v[2]), bf16_lo(v[3]), bf16_hi(v[3])};
}

// A pair's eight consecutive columns (MajorRead: the lane groups whose
// fragments have changed places).
__device__ __forceinline__ void in_order(bool swapped, const f32x4& a, const f32x4& b, f32x4& lo, f32x4& hi) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    lo[q] = swapped ? b[q] : a[q];
    hi[q] = swapped ? a[q] : b[q];
  }
}

// `rows` rows of `width` bf16 columns from row `row` on, as a buffer.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_buffer(char* base, int64_t row, int rows, int64_t width) {
  return __builtin_amdgcn_make_buffer_rsrc(base + row * width * 2, 0, static_cast<int>(rows * width * 2), 0x00020000);
}

// The tiles of a product over the experts' rows (tile_loop).
template <Product P, int BM, int BN, int BK, int WM, int WN, int STAGES>
struct RowTiles {
  static constexpr int kThreads = WM * WN * kWave;
  static constexpr int MF = BM / WM / 16, NF = BN / WN / 16;
  static constexpr bool kMajor = P == kActGrad || P == kGradX;  // weights read along their other axis
  static constexpr int kCols = P == kUp ? BN / 2 : BN;          // output columns of a tile
  using TileA = ContigTile<BM, kThreads, BK>;
  using TileB = std::conditional_t<kMajor, MajorTile<BN, kThreads, BK>, ContigTile<BN, kThreads, BK>>;
  using ReadB = std::conditional_t<kMajor, MajorRead<BN, NF, 16, true>, ContigRead<BK>>;
  static constexpr int LOADS = TileA::kLoads + TileB::kLoads;
  static constexpr bool kPaired = P != kUp || NF >= 4;  // the narrow up product has one fragment of each kind
  static constexpr int STORES = P == kUp ? MF * NF / (kPaired ? 4 : 2) : P == kActGrad ? MF * NF : MF * NF / 2;
  struct Work {
    int expert, row, rows, n0, steps, used;
  };

  const RowArgs& p;
  const ExpertTable& table;
  int row_tiles;
  char *lds_a, *lds_b;
  uint32_t at_a, at_b;
  TileA ta;
  TileB tb;
  typename TileA::Step sa;
  typename TileB::Step sb;
  const char *a0, *b0;
  uint32_t a_bytes, b_bytes;
  ContigRead<BK> ra;
  ReadB rb;
  int wm, wn;

  __device__ __forceinline__ RowTiles(const RowArgs& args, const ExpertTable& t, int mt, char* sa0, char* sb0)
      : p(args), table(t), row_tiles(mt), lds_a(sa0), lds_b(sb0) {
    at_a = lds_address(sa0);
    at_b = lds_address(sb0);
    wm = wave_id() / WN;
    wn = wave_id() % WN;
    ra.init(wm * 16);
    rb.init(wn * NF * 16);
  }

  __device__ __forceinline__ bool tile(int i, Work& w) const {
    const int at = block_tile(i, row_tiles * p.n_blocks, blockIdx.x, gridDim.x);
    if (at < 0) return false;
    // An expert's tiles lie together, so that no panel has two experts' weights.
    const int e = expert_of(table, at / p.n_blocks);
    if (e >= p.rows.E) return false;
    const int count = __builtin_amdgcn_readfirstlane(table.count[e]);
    const int mt = (count + BM - 1) / BM;
    const int mine = at - (__builtin_amdgcn_readfirstlane(table.upto[e]) - mt) * p.n_blocks;
    if (mine < 0 || mine >= mt * p.n_blocks) return false;  // counts whose sum passes 2^31, so not disjoint
    int m, n;
    panel_tile(mine, mt, p.n_blocks, m, n);
    const int in = m * BM;
    w.expert = e;
    w.row = __builtin_amdgcn_readfirstlane(table.first[e]) + in;
    w.rows = min(BM, count - in);
    w.n0 = n * kCols;
    w.steps = (p.K + BK - 1) / BK;
    w.used = (w.rows - wm * 16 + WM * 16 - 1) / (WM * 16);
    return true;
  }

  __device__ __forceinline__ void aim(const Work& w) {
    const int K = p.K, N = p.N;
    ta.init(K, [&](int r) { return r < w.rows ? r : -1; });
    a0 = p.a + static_cast<int64_t>(w.row) * K * 2;
    a_bytes = static_cast<uint32_t>(w.rows) * K * 2;
    const char* weights = p.w + w.expert * p.w_stride;
    if constexpr (kMajor) {
      b0 = weights + static_cast<int64_t>(w.n0) * 2;
      tb.init(N, N - w.n0);
    } else {
      b0 = weights + static_cast<int64_t>(w.n0) * K * 2;
      b_bytes = static_cast<uint32_t>(p.w_stride - static_cast<int64_t>(w.n0) * K * 2);
      if constexpr (P == kUp) {
        // A wave's columns are as many gate columns, then the same up columns.
        constexpr int kHalf = NF * 8;
        tb.init(K, [&](int r) {
          const int in = r % kHalf;
          const int c = r / (2 * kHalf) * kHalf + (kPaired ? paired_column(in) : in);
          return w.n0 + c < N ? c + ((r & kHalf) ? N : 0) : -1;
        });
      } else {
        tb.init(K, [&](int r) {
          const int c = paired_column(r);
          return w.n0 + c < N ? c : -1;
        });
      }
    }
  }

  __device__ __forceinline__ void begin(int step) {
    const int k0 = step * BK;
    sa = ta.step(a0, a_bytes, k0, p.K);
    if constexpr (kMajor)
      sb = tb.step(b0, p.N, k0, p.K);
    else
      sb = tb.step(b0, b_bytes, k0, p.K);
  }
  __device__ __forceinline__ void load(int i, int stage) const {
    if (i < TileA::kLoads)
      ta.load(sa, i, at_a + stage * TileA::kBytes);
    else
      tb.load(sb, i - TileA::kLoads, at_b + stage * TileB::kBytes);
  }
  __device__ __forceinline__ void read_a(int i, int stage, int h, bf16x8& f) const {
    f = ra.get(lds_a + stage * TileA::kBytes, i * WM, h);
  }
  __device__ __forceinline__ void read_b(int j, int stage, int h, bf16x8& f) const {
    f = rb.get(lds_b + stage * TileB::kBytes, j, h);
  }

  // A lane holds eight consecutive columns of one row per pair of fragments.
  __device__ __forceinline__ void store(const Work& w, const f32x4 (&acc)[NF][MF]) const {
    const int N = p.N, l = lane_id(), g = l >> 4;
    const auto out = rows_buffer(p.out, w.row, w.rows, P == kActGrad ? 2 * N : N);
    const auto gu = rows_buffer(p.gu, w.row, p.gu != nullptr ? w.rows : 0, 2 * N);
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      const int r = (i * WM + wm) * 16 + (l & 15);
      if constexpr (P == kUp && !kPaired) {
        const int c = w.n0 + wn * 16 + g * 4;
        const int at = c < N ? (r * 2 * N + c) * 2 : kOut;
        f32x4 v;
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = act_value(p.act, acc[0][i][q]) * acc[1][i][q];
        store4(out, c < N ? (r * N + c) * 2 : kOut, v);
        if (p.gu != nullptr) {
          store4(gu, at, acc[0][i]);
          store4(gu, c < N ? at + N * 2 : kOut, acc[1][i]);
        }
      } else if constexpr (P == kUp) {
#pragma unroll
        for (int j = 0; j < NF / 2; j += 2) {
          const int c = w.n0 + wn * NF * 8 + j * 16 + g * 8;
          const int at = c < N ? (r * 2 * N + c) * 2 : kOut;
          f32x4 v[2];
#pragma unroll
          for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int q = 0; q < 4; ++q)
              v[b][q] = act_value(p.act, acc[j + b][i][q]) * acc[j + b + NF / 2][i][q];
          store8(out, c < N ? (r * N + c) * 2 : kOut, v[0], v[1]);
          if (p.gu != nullptr) {
            store8(gu, at, acc[j][i], acc[j + 1][i]);
            store8(gu, c < N ? at + N * 2 : kOut, acc[j + NF / 2][i], acc[j + 1 + NF / 2][i]);
          }
        }
      } else {
        f32x4 gate[NF], up[NF];
        if constexpr (P == kActGrad) {
#pragma unroll
          for (int j = 0; j < NF; j += 2) {
            const int c = w.n0 + wn * NF * 16 + j * 16 + g * 8;
            const int at = c < N ? (r * 2 * N + c) * 2 : kOut;
            load8(gu, at, gate[j], gate[j + 1]);
            load8(gu, c < N ? at + N * 2 : kOut, up[j], up[j + 1]);
          }
        }
#pragma unroll
        for (int j = 0; j < NF; j += 2) {
          const int c = w.n0 + wn * NF * 16 + j * 16 + g * 8;
          f32x4 v[2];
          in_order(kMajor && g >= 2, acc[j][i], acc[j + 1][i], v[0], v[1]);
          if constexpr (P == kActGrad) {
            const int at = c < N ? (r * 2 * N + c) * 2 : kOut;
            f32x4 dg[2], du[2];
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                float value, slope;
                act_both(p.act, gate[j + b][q], value, slope);
                dg[b][q] = v[b][q] * up[j + b][q] * slope;
                du[b][q] = v[b][q] * value;
              }
            store8(out, at, dg[0], dg[1]);
            store8(out, c < N ? at + N * 2 : kOut, du[0], du[1]);
          } else {
            store8(out, c < N ? (r * N + c) * 2 : kOut, v[0], v[1]);
          }
        }
      }
    }
  }
};

template <Product P, int BM, int BN, int BK, int WM, int WN, int STAGES>
__global__ __launch_bounds__(WM * WN * 64) void row_product_kernel(RowArgs p) {
  using Tiles = RowTiles<P, BM, BN, BK, WM, WN, STAGES>;
  __shared__ __attribute__((aligned(1024))) char s_a[STAGES * Tiles::TileA::kBytes];
  __shared__ __attribute__((aligned(1024))) char s_b[STAGES * Tiles::TileB::kBytes];
  __shared__ ExpertTable s_table;
  const int row_tiles = fill_table(p.rows, BM, s_table);
  Tiles tiles(p, s_table, row_tiles, s_a, s_b);
  tile_loop<STAGES, BK / 32, Tiles::MF, Tiles::NF>(tiles);
}

// Weight gradients: out_e [M][N] = P_e^T Q_e over the expert's rows, P
// [rows][M], Q [rows][N].  An expert without rows gets zeros.
//
// Where the tiles of all experts are fewer than the CUs (few experts, small
// layers, many rows), each expert's rows are cut into `splits` ranges, whose
// fp32 sums go to the workspace and are added in order by a second kernel.
struct WeightArgs {
  const char* p;
  const char* q;
  char* out;
  float* partial;  // [splits][E][M][N], used when splits > 1
  ExpertRows rows;
  int M, N, m_blocks, n_blocks, splits;
};

struct WeightTile {
  int expert, split, m, n;  // m, n: tile numbers
  int row, rows;            // the split's rows
};

// Tile `mt`, `n` of the launch's (expert, split, m) x n tiles; the expert's
// rows are given.
__device__ __forceinline__ void weight_tile(const WeightArgs& p, int mt, WeightTile& t) {
  const int es = mt / p.m_blocks;
  t.m = mt - es * p.m_blocks;
  t.expert = es / p.splits;
  t.split = es - t.expert * p.splits;
}

constexpr int kRange = 64;  // ranges are whole steps

__device__ __forceinline__ void split_rows(const WeightArgs& p, int first, int all, WeightTile& t) {
  const int range = ((all + p.splits - 1) / p.splits + kRange - 1) / kRange * kRange;
  const int lo = min(all, t.split * range);
  t.row = first + lo;
  t.rows = min(range, all - lo);
}

// Four columns of one row of the result, or of this split's share of it.
__device__ __forceinline__ void store_weights_f32(const WeightArgs& p, const WeightTile& t, int m, int c, f32x4 v) {
  const bool share = p.splits > 1;
  const int64_t at = ((static_cast<int64_t>(share ? t.split : 0) * p.rows.E + t.expert) * p.M + m) * p.N + c;
  *reinterpret_cast<f32x4*>((share ? p.partial : reinterpret_cast<float*>(p.out)) + at) = v;
}

// Adds up the shares of both weight gradients (16 bytes of fp32 a thread);
// `blocks` of the launch are the first one's.
struct SumArgs {
  const float* partial;
  char* out;
  int64_t quads;  // 0: not cut into ranges
  int splits, blocks;
};

template <bool BF16>
__global__ __launch_bounds__(256) void weight_sum_kernel(SumArgs a, SumArgs b) {
  const bool second = static_cast<int>(blockIdx.x) >= a.blocks;
  const SumArgs& p = second ? b : a;
  const int64_t i = static_cast<int64_t>(blockIdx.x - (second ? a.blocks : 0)) * 256 + threadIdx.x;
  if (i >= p.quads) return;
  const f32x4* in = reinterpret_cast<const f32x4*>(p.partial);
  f32x4 v = in[i];
  for (int s = 1; s < p.splits; ++s) v += in[s * p.quads + i];
  if constexpr (BF16)
    *reinterpret_cast<bf16x4*>(p.out + i * 8) = round4(v);
  else
    *reinterpret_cast<f32x4*>(p.out + i * 16) = v;
}

// The tiles of a weight gradient (tile_loop).
template <int BM, int BN, int BK, int WM, int WN, int STAGES>
struct WeightTiles {
  static constexpr int kThreads = WM * WN * kWave;
  static constexpr int MF = BM / WM / 16, NF = BN / WN / 16;
  using TileA = MajorTile<BM, kThreads, BK>;
  using TileB = MajorTile<BN, kThreads, BK>;
  static constexpr int LOADS = TileA::kLoads + TileB::kLoads;
  static constexpr int STORES = MF * NF / 2;
  struct Work {
    WeightTile t;
    int steps, used;
  };

  const WeightArgs& p;
  const ExpertTable& table;
  int block, blocks;
  char *lds_a, *lds_b;
  uint32_t at_a, at_b;
  TileA ta;
  TileB tb;
  typename TileA::Step sa;
  typename TileB::Step sb;
  const char *a0 = nullptr, *b0 = nullptr;
  int K = 0;
  MajorRead<BM, MF, 16 * WM, false> ra;
  MajorRead<BN, NF, 16, true> rb;
  int wm, wn;

  __device__ __forceinline__ WeightTiles(const WeightArgs& args, const ExpertTable& tab, int b, int n, char* sa0,
                                         char* sb0)
      : p(args), table(tab), block(b), blocks(n), lds_a(sa0), lds_b(sb0) {
    at_a = lds_address(sa0);
    at_b = lds_address(sb0);
    wm = wave_id() / WN;
    wn = wave_id() % WN;
    ra.init(wm * 16);
    rb.init(wn * NF * 16);
  }

  __device__ __forceinline__ bool tile(int i, Work& w) const {
    const int total = p.rows.E * p.splits * p.m_blocks;
    int mt;
    if (!dealt_tile(i, total, p.n_blocks, block, blocks, mt, w.t.n)) return false;
    weight_tile(p, mt, w.t);
    split_rows(p, __builtin_amdgcn_readfirstlane(table.first[w.t.expert]),
               __builtin_amdgcn_readfirstlane(table.count[w.t.expert]), w.t);
    w.steps = (w.t.rows + BK - 1) / BK;
    w.used = (p.M - w.t.m * BM - wm * 16 + WM * 16 - 1) / (WM * 16);
    return true;
  }

  __device__ __forceinline__ void aim(const Work& w) {
    const int m0 = w.t.m * BM, n0 = w.t.n * BN;
    K = w.t.rows;
    ta.init(p.M, p.M - m0);
    tb.init(p.N, p.N - n0);
    a0 = p.p + (static_cast<int64_t>(w.t.row) * p.M + m0) * 2;
    b0 = p.q + (static_cast<int64_t>(w.t.row) * p.N + n0) * 2;
  }

  __device__ __forceinline__ void begin(int step) {
    const int k0 = step * BK;
    sa = ta.step(a0, p.M, k0, K);
    sb = tb.step(b0, p.N, k0, K);
  }
  __device__ __forceinline__ void load(int i, int stage) const {
    if (i < TileA::kLoads)
      ta.load(sa, i, at_a + stage * TileA::kBytes);
    else
      tb.load(sb, i - TileA::kLoads, at_b + stage * TileB::kBytes);
  }
  __device__ __forceinline__ void read_a(int i, int stage, int h, bf16x8& f) const {
    f = ra.get(lds_a + stage * TileA::kBytes, i, h);
  }
  __device__ __forceinline__ void read_b(int j, int stage, int h, bf16x8& f) const {
    f = rb.get(lds_b + stage * TileB::kBytes, j, h);
  }

  __device__ __forceinline__ void store(const Work& w, const f32x4 (&acc)[NF][MF]) const {
    const int l = lane_id();
    const int m0 = w.t.m * BM, n0 = w.t.n * BN;
    const bool share = p.splits > 1;
    // The tile's rows as a buffer: of the result, or of this split's share.
    const int64_t row = (static_cast<int64_t>(share ? w.t.split : 0) * p.rows.E + w.t.expert) * p.M + m0;
    const int es = share ? 4 : 2;
    const auto out = __builtin_amdgcn_make_buffer_rsrc(
        (share ? reinterpret_cast<char*>(p.partial) : p.out) + row * p.N * es, 0,
        min(BM, p.M - m0) * p.N * es, 0x00020000);
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      const int m = (i * WM + wm) * 16 + (l & 15);
#pragma unroll
      for (int j = 0; j < NF; j += 2) {
        const int c = n0 + wn * NF * 16 + j * 16 + (l >> 4) * 8;
        const int at = c < p.N ? (m * p.N + c) * es : kOut;
        f32x4 lo, hi;
        in_order(l >= 32, acc[j][i], acc[j + 1][i], lo, hi);
        if (share) {
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, lo), out, at, 0, 0);
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, hi), out, c < p.N ? at + 16 : kOut, 0, 0);
        } else {
          store8(out, at, lo, hi);
        }
      }
    }
  }
};

// Blocks [0, to_first) work on one gradient, the others on the second.
template <int BM, int BN, int BK, int WM, int WN, int STAGES>
__global__ __launch_bounds__(WM * WN * 64) void weight_product_kernel(WeightArgs first, WeightArgs second,
                                                                      int to_first) {
  using Tiles = WeightTiles<BM, BN, BK, WM, WN, STAGES>;
  __shared__ __attribute__((aligned(1024))) char s_a[STAGES * Tiles::TileA::kBytes];
  __shared__ __attribute__((aligned(1024))) char s_b[STAGES * Tiles::TileB::kBytes];
  __shared__ ExpertTable s_table;
  const int block = blockIdx.x, blocks = gridDim.x;
  const bool is_first = block < to_first;
  const WeightArgs p = is_first ? first : second;
  fill_table(p.rows, BM, s_table);
  Tiles tiles(p, s_table, is_first ? block : block - to_first, is_first ? to_first : blocks - to_first, s_a, s_b);
  tile_loop<STAGES, BK / 32, Tiles::MF, Tiles::NF>(tiles);
}

// ---------------------------------------------------------------- few rows

// One token's or a small batch's rows: a tile of 16 rows, the weights read
// once, straight into registers.  Bound by that reading: a wave has two
// batches of loads in registers, one in flight while the other is used, and
// goes from one column tile to the next without a pause in its loads.
//
// A tile of up to four rows is dot products on the vector units: a wave owns
// eight weight rows and reads 1 KiB of each at a time, lane l the k = 8 l ..
// + 7 of it.  The matrix instructions want 64 bytes of each of sixteen rows
// instead, and memory gives that at a lower rate (one token's eight experts
// of 4096 x 2048, the up product: 45 us against 50).  With more
// rows the dot products would outweigh the loads, so those tiles take MFMAs:
// the block's four waves share 32 weight rows (16 gate and 16 up rows of the
// same columns, or 32 columns of y) and a quarter of K each, and their sums
// meet in LDS.
constexpr int kFewRows = 16;
constexpr int kDotRows = 4;
constexpr int kFewCols = 32;
constexpr int kAhead = 4;
constexpr int kFewK = 32;  // k of one MFMA

// The dot products of a tile of at most kDotRows rows over column tiles
// [tile, last).  Wave w has columns 4 w .. + 3 of a tile's 16 (gate and up
// rows of each), or 8 w .. + 7 of its 32.
constexpr int kDotK = kWave * 8;

struct DotBatch {
  u32x4 w[8], x[kDotRows];
};

template <Product P>
__device__ __forceinline__ void dot_tiles(const RowArgs& p, const RowTile& t, int tile, int last) {
  const int K = p.K, N = p.N;
  const int l = lane_id(), w = wave_id();
  constexpr int kCols = P == kUp ? 16 : kFewCols;
  const char* wt = p.w + t.expert * p.w_stride;
  const char* a0 = p.a + static_cast<int64_t>(t.row) * K * 2;
  const int steps = (K + kDotK - 1) / kDotK;
  const u32x4 zero = {0, 0, 0, 0};
  // Weight row q of this wave: column and half of it.
  auto column = [&](int tile, int q) { return tile * kCols + (P == kUp ? w * 4 + (q & 3) : w * 8 + q); };
  auto load = [&](int tile, int step, DotBatch& f) {
    const int k = step * kDotK + l * 8;
    const bool in = k < K;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int c = column(tile, q);
      const char* row = wt + static_cast<int64_t>(P == kUp && q >= 4 ? N + c : c) * K * 2;
      f.w[q] = in && c < N ? __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(row) + k / 8) : zero;
    }
#pragma unroll
    for (int r = 0; r < kDotRows; ++r)
      f.x[r] = in && r < t.rows
          ? *reinterpret_cast<const u32x4*>(a0 + (static_cast<int64_t>(r) * K + k) * 2) : zero;
  };
  float acc[kDotRows][8] = {};
  auto multiply = [&](const DotBatch& f) {
#pragma unroll
    for (int r = 0; r < kDotRows; ++r) {
      if (r >= t.rows) break;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float lo = bf16_lo(f.x[r][i]), hi = bf16_hi(f.x[r][i]);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          acc[r][q] = __builtin_fmaf(bf16_lo(f.w[q][i]), lo, acc[r][q]);
          acc[r][q] = __builtin_fmaf(bf16_hi(f.w[q][i]), hi, acc[r][q]);
        }
      }
    }
  };
  // Sums over the lanes; lane 8 r + q then has weight row q for row r.
  auto finish = [&](int tile) {
    float mine = 0.f;
#pragma unroll
    for (int r = 0; r < kDotRows; ++r) {
      if (r >= t.rows) break;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float sum = wave_sum_f(acc[r][q]);
        if (l == r * 8 + q) mine = sum;
        acc[r][q] = 0.f;
      }
    }
    const int r = l >> 3, q = l & 7;
    const int c = column(tile, q);
    const int64_t row = t.row + r;
    __bf16* out = reinterpret_cast<__bf16*>(p.out);
    if constexpr (P == kUp) {
      const float up = __shfl(mine, l + 4, kWave);
      if (r >= t.rows || c >= N) return;
      if (q < 4) out[row * N + c] = static_cast<__bf16>(act_value(p.act, mine) * up);
      if (p.gu != nullptr)
        reinterpret_cast<__bf16*>(p.gu)[row * 2 * N + (q < 4 ? 0 : N) + c] = static_cast<__bf16>(mine);
    } else {
      if (r < t.rows && c < N) out[row * N + c] = static_cast<__bf16>(mine);
    }
  };
  DotBatch f[2];
  load(tile, 0, f[0]);
  int step = 0;
  for (bool more = true; more;) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      // The next batch: of this tile, or the first of the next one.
      const bool ends = step + 1 == steps;
      const int next_tile = ends ? tile + 1 : tile, next_step = ends ? 0 : step + 1;
      more = next_tile < last;
      if (more) load(next_tile, next_step, f[u ^ 1]);
      multiply(f[u]);
      if (ends) finish(tile);
      tile = next_tile;
      step = next_step;
      if (!more) break;
    }
  }
}

struct FewBatch {
  u32x4 x[kAhead], w0[kAhead], w1[kAhead];
};

template <Product P>
__global__ __launch_bounds__(256) void few_rows_kernel(RowArgs p) {
  static_assert(P == kUp || P == kDown, "the forward products");
  __shared__ f32x4 s_acc[2][4][2][kWave];
  RowTile t;
  int nb;
  if (!find_tile(p.rows, blockIdx.x, kFewRows, p.n_blocks, reinterpret_cast<char*>(s_acc), t, nb)) return;
  const int K = p.K, N = p.N;
  const int l = lane_id(), w = wave_id();
  constexpr int kCols = P == kUp ? 16 : kFewCols;
  const int tiles = (N + kCols - 1) / kCols;
  int tile = nb * p.n_per;
  const int last = min(tiles, tile + p.n_per);
  if (t.rows <= kDotRows) {
    dot_tiles<P>(p, t, tile, last);
    return;
  }
  const char* wt = p.w + t.expert * p.w_stride;
  const bool in_a = (l & 15) < t.rows;
  // Wave w takes batches [w, w + 1) * batches / 4 of the K loop.
  constexpr int kBatch = kAhead * kFewK;
  const int batches = (K + kBatch - 1) / kBatch;
  const int per = (batches + 3) / 4;
  const int k_first = w * per * kBatch;
  const int k_end = min(K, k_first + per * kBatch);
  const char* a0 = p.a + static_cast<int64_t>(t.row + (in_a ? (l & 15) : 0)) * K * 2;

  // Batch b of the block's column tiles, in order: tile b / per, k batch b % per.
  auto load = [&](int tile, int batch, FewBatch& f) {
    // This lane's weight rows: column l % 16 of the gate and the up half, or
    // of both halves of the 32 columns.
    const int c0 = tile * kCols + (l & 15), c1 = P == kUp ? c0 : c0 + 16;
    const bool in0 = c0 < N, in1 = c1 < N;
    const char* b0 = wt + static_cast<int64_t>(in0 ? c0 : 0) * K * 2;
    const char* b1 = wt + static_cast<int64_t>(in1 ? (P == kUp ? N + c1 : c1) : 0) * K * 2;
    const u32x4 zero = {0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < kAhead; ++s) {
      const int k = k_first + batch * kBatch + s * kFewK + (l >> 4) * 8;
      const bool in = k < k_end;
      const int64_t at = static_cast<int64_t>(k) * 2;
      f.w0[s] = in && in0 ? __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(b0 + at)) : zero;
      f.w1[s] = in && in1 ? __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(b1 + at)) : zero;
      f.x[s] = in && in_a ? *reinterpret_cast<const u32x4*>(a0 + at) : zero;
    }
  };
  f32x4 acc0 = {0, 0, 0, 0}, acc1 = {0, 0, 0, 0};
  auto multiply = [&](const FewBatch& f) {
#pragma unroll
    for (int s = 0; s < kAhead; ++s) {
      const bf16x8 xa = __builtin_bit_cast(bf16x8, f.x[s]);
      acc0 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, f.w0[s]), xa, acc0, 0, 0, 0);
      acc1 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, f.w1[s]), xa, acc1, 0, 0, 0);
    }
  };
  // The four waves' sums of a column tile, and its outputs.  The LDS buffer
  // alternates: it is written again two tiles on, past the next barrier.
  auto finish = [&](int tile) {
    f32x4(*part)[2][kWave] = s_acc[tile & 1];
    part[w][0][l] = acc0;
    part[w][1][l] = acc1;
    acc0 = acc1 = f32x4{0, 0, 0, 0};
    __syncthreads();
    const int r = l & 15;
    const int64_t row = t.row + r;
    const int n0 = tile * kCols;
    if constexpr (P == kUp) {
      const int c = n0 + (l >> 4) * 4;
      if (w != (tile & 3) || r >= t.rows || c >= N) return;  // the waves in turn
      f32x4 g = part[0][0][l], u = part[0][1][l];
#pragma unroll
      for (int i = 1; i < 4; ++i) {
        g += part[i][0][l];
        u += part[i][1][l];
      }
      f32x4 v;
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = act_value(p.act, g[q]) * u[q];
      *reinterpret_cast<bf16x4*>(p.out + (row * N + c) * 2) = round4(v);
      if (p.gu != nullptr) {
        *reinterpret_cast<bf16x4*>(p.gu + (row * 2 * N + c) * 2) = round4(g);
        *reinterpret_cast<bf16x4*>(p.gu + (row * 2 * N + N + c) * 2) = round4(u);
      }
    } else {
      const int half = (w + tile) & 3;
      const int c = n0 + half * 16 + (l >> 4) * 4;
      if (half >= 2 || r >= t.rows || c >= N) return;
      f32x4 v = part[0][half][l];
#pragma unroll
      for (int i = 1; i < 4; ++i) v += part[i][half][l];
      *reinterpret_cast<bf16x4*>(p.out + (row * N + c) * 2) = round4(v);
    }
  };

  FewBatch f[2];
  load(tile, 0, f[0]);
  int batch = 0;
  for (bool more = true; more;) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      // The next batch: of this tile, or the first of the next one.
      const bool ends = batch + 1 == per;
      const int next_tile = ends ? tile + 1 : tile, next_batch = ends ? 0 : batch + 1;
      more = next_tile < last;
      if (more) load(next_tile, next_batch, f[u ^ 1]);
      multiply(f[u]);
      if (ends) finish(tile);
      tile = next_tile;
      batch = next_batch;
      if (!more) break;
    }
  }
}

// ---------------------------------------------------------------- fp32 tiles

// fp32 rows and weights: the same products on v_mfma_f32_16x16x4_f32.  Four
// waves of 16 MF x 16 NF make a tile of 32 MF x 32 NF; K goes in steps of FK
// through registers into two LDS buffers, an operand in the order of its
// memory: [row][k], its chunks of four k permuted by the row, or [k][column]
// with rows 4 floats longer than the tile.  Lane group g takes k = 4 g + q of
// every 16 in the q-th MFMA, so that a fragment of the first kind is one
// 16-byte read; both kinds of read fall on different banks.  Small layers take
// small tiles, which fill the chip, and long steps, since each step's loads
// are a memory latency to wait for.  8 experts of 2048 x 1024, 4096 rows each:
// 3.56 ms forward, 116 TFLOP/s (a library product of 8192 reaches 147); rows
// padded by four floats instead of permuted chunks: 3.73.
//
// One operand tile of T rows (CONTIG: k contiguous) or columns (K major).
template <int T, int FK, bool CONTIG>
struct FloatTile {
  static_assert(FK == 32 || FK == 64, "the chunk permutation");
  static constexpr int kStride = CONTIG ? FK : T + 4;
  static constexpr int kFloats = (CONTIG ? T : FK) * kStride;
  static constexpr int kLoads = T * FK / 4 / 256;
  f32x4 v[kLoads];
  // Where chunk c (four k) of row r lies in the row (CONTIG).
  __device__ __forceinline__ static int chunk_at(int r, int c) {
    return c ^ (FK == 64 ? 2 * (r & 7) : (r >> 1) & 7);
  }
  // row(r): pointer to tile row r's first k (CONTIG), or null;
  // else base: tile column 0 at k = 0, ld its row length, cols valid columns.
  template <class Row>
  __device__ __forceinline__ void fetch(Row row, const float* base, int64_t ld, int cols, int k0, int K) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int id = i * 256 + threadIdx.x;
      v[i] = f32x4{0.f, 0.f, 0.f, 0.f};
      if constexpr (CONTIG) {
        const int k = k0 + (id % (FK / 4)) * 4;
        const float* p = row(id / (FK / 4));
        if (p != nullptr && k < K) v[i] = *reinterpret_cast<const f32x4*>(p + k);
      } else {
        const int k = k0 + id / (T / 4), c = id % (T / 4) * 4;
        if (k < K && c < cols) v[i] = *reinterpret_cast<const f32x4*>(base + k * ld + c);
      }
    }
  }
  __device__ __forceinline__ void store(float* s) const {
    constexpr int kQuads = (CONTIG ? FK : T) / 4;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int id = i * 256 + threadIdx.x;
      const int r = id / kQuads, c = id % kQuads;
      *reinterpret_cast<f32x4*>(s + r * kStride + (CONTIG ? chunk_at(r, c) : c) * 4) = v[i];
    }
  }
  // k = k0 + 4 (lane / 16) .. + 3 of tile row or column at + lane % 16.
  __device__ __forceinline__ static f32x4 read(const float* s, int k0, int at) {
    const int g = lane_id() >> 4, r = at + (lane_id() & 15);
    if constexpr (CONTIG)
      return *reinterpret_cast<const f32x4*>(s + r * kStride + chunk_at(r, k0 / 4 + g) * 4);
    f32x4 f;
#pragma unroll
    for (int q = 0; q < 4; ++q) f[q] = s[(k0 + 4 * g + q) * kStride + r];
    return f;
  }
};

// acc[j][i]: 16 columns (rows of operand b) j by 16 rows i of the wave.  Two
// sums of half the k each, added at the end: half the roundings in a row.
template <int MF, int NF, int FK, bool A_CONTIG, bool B_CONTIG>
constexpr int kFloatLds = 2 * (FloatTile<32 * MF, FK, A_CONTIG>::kFloats + FloatTile<32 * NF, FK, B_CONTIG>::kFloats);

template <int MF, int NF, int FK, bool A_CONTIG, bool B_CONTIG, class RowA, class RowB>
__device__ __forceinline__ void float_loop(float* lds, int K, RowA row_a, const float* a0, int64_t lda, int cols_a,
                                           RowB row_b, const float* b0, int64_t ldb, int cols_b,
                                           f32x4 (&acc)[NF][MF]) {
  using TA = FloatTile<32 * MF, FK, A_CONTIG>;
  using TB = FloatTile<32 * NF, FK, B_CONTIG>;
  TA ta;
  TB tb;
  f32x4 odd[NF][MF] = {};
  const int ra = wave_id() / 2 * 16 * MF, rb = wave_id() % 2 * 16 * NF;
  ta.fetch(row_a, a0, lda, cols_a, 0, K);
  tb.fetch(row_b, b0, ldb, cols_b, 0, K);
  int buf = 0;
  for (int k0 = 0; k0 < K; k0 += FK, buf ^= 1) {
    float* s_a = lds + buf * TA::kFloats;
    float* s_b = lds + 2 * TA::kFloats + buf * TB::kFloats;
    ta.store(s_a);
    tb.store(s_b);
    __syncthreads();
    if (k0 + FK < K) {
      ta.fetch(row_a, a0, lda, cols_a, k0 + FK, K);
      tb.fetch(row_b, b0, ldb, cols_b, k0 + FK, K);
    }
#pragma unroll
    for (int k = 0; k < FK; k += 16) {
      f32x4 fa[MF], fb[NF];
#pragma unroll
      for (int i = 0; i < MF; ++i) fa[i] = TA::read(s_a, k, ra + i * 16);
#pragma unroll
      for (int j = 0; j < NF; ++j) fb[j] = TB::read(s_b, k, rb + j * 16);
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int i = 0; i < MF; ++i)
#pragma unroll
          for (int j = 0; j < NF; ++j) {
            f32x4& sum = (q & 1) ? odd[j][i] : acc[j][i];
            sum = __builtin_amdgcn_mfma_f32_16x16x4f32(fb[j][q], fa[i][q], sum, 0, 0, 0);
          }
    }
  }
#pragma unroll
  for (int j = 0; j < NF; ++j)
#pragma unroll
    for (int i = 0; i < MF; ++i) acc[j][i] += odd[j][i];
}

template <Product P>
constexpr bool kReadsMajor = P == kActGrad || P == kGradX;

// Block `block` of a product over the experts' rows.
template <Product P, int MF, int NF, int FK>
__device__ __forceinline__ void row_block_f32(const RowArgs& p, int block, float* lds) {
  constexpr int TN = 32 * NF;
  constexpr bool kMajor = kReadsMajor<P>;
  RowTile t;
  int nt;
  if (!find_tile(p.rows, block, 32 * MF, p.n_blocks, reinterpret_cast<char*>(lds), t, nt)) return;
  const int K = p.K, N = p.N;
  constexpr int kCols = P == kUp ? TN / 2 : TN;
  const int n0 = nt * kCols;
  const float* a0 = reinterpret_cast<const float*>(p.a) + static_cast<int64_t>(t.row) * K;
  const float* w = reinterpret_cast<const float*>(p.w + t.expert * p.w_stride);
  auto row_a = [&](int r) { return r < t.rows ? a0 + static_cast<int64_t>(r) * K : nullptr; };
  // kUp: a wave's 16 NF columns are 8 NF gate columns and the same up ones,
  // in turns of 16.
  auto row_b = [&](int r) -> const float* {
    if constexpr (P == kUp) {
      const int c = n0 + r / 32 * 16 + r % 16;
      return c < N ? w + static_cast<int64_t>((r & 16) ? N + c : c) * K : nullptr;
    } else {
      return n0 + r < N ? w + static_cast<int64_t>(n0 + r) * K : nullptr;
    }
  };
  f32x4 acc[NF][MF] = {};
  float_loop<MF, NF, FK, true, !kMajor>(lds, K, row_a, a0, K, 0, row_b, w + n0, N, N - n0, acc);

  const int l = lane_id();
  float* out = reinterpret_cast<float*>(p.out);
  float* gu = reinterpret_cast<float*>(p.gu);
#pragma unroll
  for (int i = 0; i < MF; ++i) {
    const int r = wave_id() / 2 * 16 * MF + i * 16 + (l & 15);
    if (r >= t.rows) continue;
    const int64_t row = t.row + r;
    if constexpr (P == kUp) {
#pragma unroll
      for (int j = 0; j < NF; j += 2) {
        const int c = n0 + wave_id() % 2 * 8 * NF + j * 8 + (l >> 4) * 4;
        if (c >= N) continue;
        f32x4 v;
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = act_value(p.act, acc[j][i][q]) * acc[j + 1][i][q];
        *reinterpret_cast<f32x4*>(out + row * N + c) = v;
        if (gu != nullptr) {
          *reinterpret_cast<f32x4*>(gu + row * 2 * N + c) = acc[j][i];
          *reinterpret_cast<f32x4*>(gu + row * 2 * N + N + c) = acc[j + 1][i];
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < NF; ++j) {
        const int c = n0 + wave_id() % 2 * 16 * NF + j * 16 + (l >> 4) * 4;
        if (c >= N) continue;
        if constexpr (P == kActGrad) {
          const f32x4 g = *reinterpret_cast<const f32x4*>(gu + row * 2 * N + c);
          const f32x4 u = *reinterpret_cast<const f32x4*>(gu + row * 2 * N + N + c);
          f32x4 dg, du;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float value, slope;
            act_both(p.act, g[q], value, slope);
            dg[q] = acc[j][i][q] * u[q] * slope;
            du[q] = acc[j][i][q] * value;
          }
          *reinterpret_cast<f32x4*>(out + row * 2 * N + c) = dg;
          *reinterpret_cast<f32x4*>(out + row * 2 * N + N + c) = du;
        } else {
          *reinterpret_cast<f32x4*>(out + row * N + c) = acc[j][i];
        }
      }
    }
  }
}

template <Product P, int MF, int NF, int FK>
__global__ __launch_bounds__(256) void row_product_f32_kernel(RowArgs p) {
  __shared__ __attribute__((aligned(16))) float s_lds[kFloatLds<MF, NF, FK, true, !kReadsMajor<P>>];
  row_block_f32<P, MF, NF, FK>(p, blockIdx.x, s_lds);
}

// Block `block` of a weight gradient.
template <int MF, int NF, int FK>
__device__ __forceinline__ void weight_block_f32(const WeightArgs& p, int block, float* lds) {
  WeightTile t;
  int mt, first;
  if (!tile_of(block, p.rows.E * p.splits * p.m_blocks, p.n_blocks, mt, t.n)) return;
  weight_tile(p, mt, t);
  const int all = __builtin_amdgcn_readfirstlane(rows_of(p.rows, t.expert, first));
  split_rows(p, __builtin_amdgcn_readfirstlane(first), all, t);
  const int m0 = t.m * 32 * MF, n0 = t.n * 32 * NF;
  const int M = p.M, N = p.N;
  const float* a0 = reinterpret_cast<const float*>(p.p) + static_cast<int64_t>(t.row) * M + m0;
  const float* b0 = reinterpret_cast<const float*>(p.q) + static_cast<int64_t>(t.row) * N + n0;
  auto none = [](int) -> const float* { return nullptr; };
  f32x4 acc[NF][MF] = {};
  float_loop<MF, NF, FK, false, false>(lds, t.rows, none, a0, M, M - m0, none, b0, N, N - n0, acc);
  const int l = lane_id();
#pragma unroll
  for (int i = 0; i < MF; ++i) {
    const int m = m0 + wave_id() / 2 * 16 * MF + i * 16 + (l & 15);
    if (m >= M) continue;
#pragma unroll
    for (int j = 0; j < NF; ++j) {
      const int c = n0 + wave_id() % 2 * 16 * NF + j * 16 + (l >> 4) * 4;
      if (c < N) store_weights_f32(p, t, m, c, acc[j][i]);
    }
  }
}

template <int MF, int NF, int FK>
__global__ __launch_bounds__(256) void weight_product_f32_kernel(WeightArgs p) {
  __shared__ __attribute__((aligned(16))) float s_lds[kFloatLds<MF, NF, FK, false, false>];
  weight_block_f32<MF, NF, FK>(p, blockIdx.x, s_lds);
}

// What follows [dg | du] in the backward of a small layer, in one launch: the
// three products need nothing of each other, and each alone leaves most of the
// chip idle.  Blocks [0, to_in) form dWin, [to_in, to_down) dWdown, the rest dx.
template <int MF, int NF, int FK>
__global__ __launch_bounds__(256) void gradients_f32_kernel(WeightArgs in, WeightArgs down, RowArgs dx, int to_in,
                                                            int to_down) {
  constexpr int kWeights = kFloatLds<MF, NF, FK, false, false>, kRows = kFloatLds<MF, NF, FK, true, false>;
  __shared__ __attribute__((aligned(16))) float s_lds[kWeights > kRows ? kWeights : kRows];
  const int block = blockIdx.x;
  if (block < to_in)
    weight_block_f32<MF, NF, FK>(in, block, s_lds);
  else if (block < to_down)
    weight_block_f32<MF, NF, FK>(down, block - to_in, s_lds);
  else
    row_block_f32<kGradX, MF, NF, FK>(dx, block - to_down, s_lds);
}

// ---------------------------------------------------------------- launches

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int kCus = 256;
constexpr int kFewPerCu = 8;

// A product over the experts' rows, with the tile that the rows an expert
// has on average fill.
template <Product P, int BM, int BN, int BK, int WM, int WN, int STAGES>
int launch_rows(RowArgs p, hipStream_t s) {
  p.n_blocks = static_cast<int>(ceil_div(p.N, P == kUp ? BN / 2 : BN));
  const int64_t tiles = most_tiles(p.rows.R, p.rows.E, BM) * p.n_blocks;
  if (tiles > INT32_MAX) return MOE_ERR_SHAPE;
  // As many blocks as are resident at once (160 KB of LDS a CU).
  constexpr int64_t kResident = kCus * (160 * 1024 / (STAGES * (BM + BN) * BK * 2 + 4096));
  const int64_t blocks = ceil_div(tiles < kResident ? tiles : kResident, kXcds) * kXcds;
  row_product_kernel<P, BM, BN, BK, WM, WN, STAGES><<<static_cast<unsigned>(blocks), WM * WN * kWave, 0, s>>>(p);
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}

// Column tiles a block: one while there are at most eight blocks a CU (two are
// resident), then as many as keep it so; a block's start (finding
// its rows, the first loads) is then paid once.
template <Product P>
int launch_few(RowArgs p, hipStream_t s) {
  const int64_t tiles = ceil_div(p.N, P == kUp ? 16 : kFewCols);
  const int64_t mt = most_tiles(p.rows.R, p.rows.E, kFewRows);
  const int64_t per = mt * tiles / (kCus * kFewPerCu);
  p.n_per = static_cast<int>(per < 1 ? 1 : per > tiles ? tiles : per);
  p.n_blocks = static_cast<int>(ceil_div(tiles, p.n_per));
  const int64_t blocks = ceil_div(mt * p.n_blocks, kXcds) * kXcds;
  if (!grid_ok(blocks, 256)) return MOE_ERR_SHAPE;
  few_rows_kernel<P><<<static_cast<unsigned>(blocks), 256, 0, s>>>(p);
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}

template <Product P, int MF, int NF, int FK>
int launch_rows_f32(RowArgs p, hipStream_t s) {
  constexpr int TN = 32 * NF;
  p.n_blocks = static_cast<int>(ceil_div(p.N, P == kUp ? TN / 2 : TN));
  const int64_t blocks = ceil_div(most_tiles(p.rows.R, p.rows.E, 32 * MF) * p.n_blocks, kXcds) * kXcds;
  if (!grid_ok(blocks, 256)) return MOE_ERR_SHAPE;
  row_product_f32_kernel<P, MF, NF, FK><<<static_cast<unsigned>(blocks), 256, 0, s>>>(p);
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}

// The fp32 tile of a product of `rows` x `cols` outputs (over all experts): 64
// x 64 where that makes two blocks a CU or more, else 32 x 64.  8 experts of
// 256 x 256, 512 rows each: 64 us backward by this rule, 73 with 64 x 64
// already from one block a CU; 8 of 1024 x 1024, 1024 rows: 513 us forward
// with 64 x 64, 556 with 32 x 64 (and 679 with 128 x 128: three times the
// registers, one block a CU).
inline int f32_tile(int64_t rows, int64_t cols) {
  return rows / 64 * ceil_div(cols, 64) >= 2 * kCus ? 64 : 32;
}

// Which tile, measured on MI355X (bf16, time of forward / backward):
//  - up to one row an expert on average: the few-rows kernel (rows routed at
//    random, forward: 64 experts of 4096 x 2048, 48 rows in all 288 us, tiles
//    of 128 346 side by side (280 to 320 by routing and card); 8 of 4096 x 8192, 8 rows 176 and 247; with two rows an
//    expert 546 and 476, 286 and 282);
//  - from 512 rows an expert, with a tile for half the CUs: 256 x 256, fewest
//    bytes a product (64 experts of 4096 x 2048, 1024 rows: 3.19 / 6.34 ms
//    against 3.40 / 6.81 with 128 x 256; 8 of 2048 x 1024, 512 rows: 79 / 171
//    us against 92 / 182; below, the narrower tile's smaller rounding up wins:
//    64 of 2048 x 1024, 320 rows: 350 / 774 against 389 / 826);
//  - fewer tiles than half the CUs: 128 x 64, two blocks a CU (one expert of
//    2160 x 400, 374 rows: 25 / 46 us against 41 / 68 with 128 x 256; 8 of
//    2048 x 1024, 64 rows: 28 / 70 against 43 / 96).
// A weight read along its other axis, whose lines are whole in any step, goes
// in steps of 32 k, four in LDS (64 experts of 4096 x 2048, 65536 rows, the
// backward: 6.34 ms against 6.42 in steps of 64); K-contiguous operands in
// steps of 64.
template <Product P>
int row_product(const RowArgs& p, int dtype, hipStream_t s) {
  const int64_t R = p.rows.R, E = p.rows.E;
  if (dtype == MOE_F32) {
    const int tile = f32_tile(R, P == kUp ? 2 * static_cast<int64_t>(p.N) : p.N);
    return tile == 64 ? launch_rows_f32<P, 2, 2, 32>(p, s) : launch_rows_f32<P, 1, 2, 64>(p, s);
  }
  if constexpr (P == kUp || P == kDown)
    if (R <= E) return launch_few<P>(p, s);
  const int64_t cols = P == kUp ? 2 * static_cast<int64_t>(p.N) : p.N;
  if (R >= 512 * E && R / 256 * ceil_div(cols, 256) >= kCus / 2) {
    if constexpr (P == kUp || P == kDown) return launch_rows<P, 256, 256, 64, 2, 4, 2>(p, s);
    return launch_rows<P, 256, 256, 32, 2, 4, 4>(p, s);
  }
  if (most_tiles(R, p.rows.E, 128) * ceil_div(cols, 256) >= kCus / 2)
    return launch_rows<P, 128, 256, 64, 2, 4, 3>(p, s);
  return launch_rows<P, 128, 64, 64, 4, 2, 3>(p, s);
}

// The tile of a weight gradient and the ranges its rows are cut into: where
// the tiles are fewer than the CUs, as many as make the shortest time of a
// block that walks its range and a second launch that adds the shares up.
// The constants are measured (bf16, backward in all: 4 experts of 728 x 200,
// 28000 rows each: 1306 us uncut, 349 cut; 8 of 512 x 512, 4096 rows: 316 and
// 237; 8 of 1024 x 512, 512 rows: 77 uncut, 102 in two ranges, whose shares
// cost more than they save).
constexpr double kRowUs = 0.023;          // one row of a tile
constexpr double kSumUs = 3.0;            // the second launch
constexpr double kShareUs = 8.0 / 5.0e6;  // an element of a share, written and read

struct WeightPlan {
  int tm, tn, threads, splits;
  int64_t partial_bytes;
};

WeightPlan weight_plan(int64_t R, int E, int64_t M, int64_t N, int dtype) {
  WeightPlan w = {256, 256, 512, 1, 0};
  if (dtype == MOE_F32) {
    w.tm = f32_tile(E * M, N);
    w.tn = 64;
    w.threads = 256;
  }
  const int64_t blocks = E * ceil_div(M, w.tm) * ceil_div(N, w.tn);
  const double rows = static_cast<double>(R) / E;
  double least = rows * kRowUs;
  for (int64_t n = 2; n <= kCus / blocks; ++n) {
    const double us = rows / n * kRowUs + kSumUs + static_cast<double>(n * E * M * N) * kShareUs;
    if (us < least) {
      least = us;
      w.splits = static_cast<int>(n);
    }
  }
  if (w.splits > 1) w.partial_bytes = w.splits * E * M * N * 4;
  return w;
}

// Fills in a gradient's tiles; returns their number.
int64_t plan_weights(WeightArgs& p, const WeightPlan& w) {
  p.m_blocks = static_cast<int>(ceil_div(p.M, w.tm));
  p.n_blocks = static_cast<int>(ceil_div(p.N, w.tn));
  p.splits = w.splits;
  return static_cast<int64_t>(p.rows.E) * w.splits * p.m_blocks * p.n_blocks;
}

int weight_product_f32(WeightArgs p, const WeightPlan& w, hipStream_t s) {
  const int64_t blocks = ceil_div(plan_weights(p, w), kXcds) * kXcds;
  if (!grid_ok(blocks, w.threads)) return MOE_ERR_SHAPE;
  auto kernel = w.tm == 64 ? weight_product_f32_kernel<2, 2, 32> : weight_product_f32_kernel<1, 2, 64>;
  kernel<<<static_cast<unsigned>(blocks), w.threads, 0, s>>>(p);
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}

// Both weight gradients: in one launch where their tiles together are no more
// than the CUs (8 experts of 1024 x 512, 1024 rows each, the whole backward: 85
// us against 114 in two), else one after the other, a block a CU.
int weight_products(WeightArgs in, WeightArgs down, const WeightPlan& w, const WeightPlan& w_down, hipStream_t s) {
  constexpr auto kernel = weight_product_kernel<256, 256, 32, 2, 4, 4>;
  const int64_t tiles[2] = {plan_weights(in, w), plan_weights(down, w_down)};
  if (tiles[0] > INT32_MAX || tiles[1] > INT32_MAX) return MOE_ERR_SHAPE;
  int blocks[2];
  for (int i = 0; i < 2; ++i)
    blocks[i] = static_cast<int>(ceil_div(tiles[i] < kCus ? tiles[i] : kCus, kXcds) * kXcds);
  if (blocks[0] + blocks[1] <= kCus) {
    kernel<<<blocks[0] + blocks[1], w.threads, 0, s>>>(in, down, blocks[0]);
    MOE_CHECK_LAUNCH();
  } else {
    kernel<<<blocks[0], w.threads, 0, s>>>(in, in, blocks[0]);
    MOE_CHECK_LAUNCH();
    kernel<<<blocks[1], w.threads, 0, s>>>(down, down, blocks[1]);
    MOE_CHECK_LAUNCH();
  }
  return MOE_OK;
}

SumArgs sum_args(const WeightArgs& p, const WeightPlan& w) {
  SumArgs a = {p.partial, p.out, 0, w.splits, 0};
  if (w.splits > 1) {
    a.quads = static_cast<int64_t>(p.rows.E) * p.M * p.N / 4;
    a.blocks = static_cast<int>(ceil_div(a.quads, 256));
  }
  return a;
}

int sum_shares(const SumArgs& a, const SumArgs& b, int dtype, hipStream_t s) {
  if (a.blocks + b.blocks == 0) return MOE_OK;
  auto kernel = dtype == MOE_BF16 ? weight_sum_kernel<true> : weight_sum_kernel<false>;
  kernel<<<static_cast<unsigned>(a.blocks + b.blocks), 256, 0, s>>>(a, b);
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}

// dx and both weight gradients, from [dg | du].  fp32 products that all take
// the small tile go out together (8 experts of 128 x 96, 512 rows each, the
// whole backward: 22 us against 34 with a launch each).
int gradients(const RowArgs& dx, WeightArgs in, WeightArgs down, const WeightPlan& plan_in,
              const WeightPlan& plan_down, int dtype, hipStream_t s) {
  const int64_t R = dx.rows.R;
  const int64_t tiles_in = ceil_div(plan_weights(in, plan_in), kXcds) * kXcds;
  const int64_t tiles_down = ceil_div(plan_weights(down, plan_down), kXcds) * kXcds;
  const int64_t tiles_x = ceil_div(most_tiles(R, dx.rows.E, 32) * ceil_div(dx.N, 64), kXcds) * kXcds;
  if (dtype == MOE_F32 && plan_in.tm == 32 && plan_down.tm == 32 && f32_tile(R, dx.N) == 32 && R > 0) {
    const int64_t blocks = tiles_in + tiles_down + tiles_x;
    if (!grid_ok(blocks, 256)) return MOE_ERR_SHAPE;
    RowArgs x = dx;
    x.n_blocks = static_cast<int>(ceil_div(dx.N, 64));
    gradients_f32_kernel<1, 2, 64><<<static_cast<unsigned>(blocks), 256, 0, s>>>(
        in, down, x, static_cast<int>(tiles_in), static_cast<int>(tiles_in + tiles_down));
    MOE_CHECK_LAUNCH();
  } else {
    if (R > 0)
      if (const int st = row_product<kGradX>(dx, dtype, s)) return st;
    if (dtype == MOE_F32) {
      if (const int st = weight_product_f32(in, plan_in, s)) return st;
      if (const int st = weight_product_f32(down, plan_down, s)) return st;
    } else if (const int st = weight_products(in, down, plan_in, plan_down, s)) {
      return st;
    }
  }
  return sum_shares(sum_args(in, plan_in), sum_args(down, plan_down), dtype, s);
}

// The backward's workspace: [dg | du], then the shares of dWin and of dWdown.
struct BackwardSpace {
  int64_t in, down, all;  // offsets, and the size
};

BackwardSpace backward_space(int64_t R, int64_t F, int dtype, const WeightPlan& in, const WeightPlan& down) {
  BackwardSpace b;
  b.in = (R * 2 * F * (dtype == MOE_BF16 ? 2 : 4) + 255) / 256 * 256;
  b.down = b.in + (in.partial_bytes + 255) / 256 * 256;
  b.all = b.down + down.partial_bytes;
  return b;
}

int ffn_check(int64_t R, int64_t H, int64_t F, int E, int dtype, int act) {
  if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_ERR_DTYPE;
  if (act != MOE_ACT_SILU && act != MOE_ACT_GELU) return MOE_ERR_DTYPE;
  const int64_t es = dtype == MOE_BF16 ? 2 : 4;
  // One expert's projections, and a tile's rows, are addressed through
  // 32-bit byte offsets; rows are counted in 32 bits and rounded up to whole
  // tiles and ranges (of 256 at most).
  if (R < 0 || R > INT32_MAX - 511 || E < 1 || E > MOE_MAX_E || H <= 0 || F <= 0 || H > (1 << 21) ||
      F > (1 << 20) || 2 * F * H * es >= kOut)
    return MOE_ERR_SHAPE;
  if (H * es % 16 != 0 || F * es % 16 != 0) return MOE_ERR_ALIGN;
  return MOE_OK;
}

bool aligned16(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (reinterpret_cast<uintptr_t>(p) % 16 != 0) return false;
  return true;
}

struct Span {
  const void* p;
  int64_t bytes;
};

// True when an output shares bytes with an input or another output.
bool any_overlap(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  for (const Span* o = outs.begin(); o != outs.end(); ++o) {
    for (const Span& i : ins)
      if (overlap(o->p, o->bytes, i.p, i.bytes)) return true;
    for (const Span* q = o + 1; q != outs.end(); ++q)
      if (overlap(o->p, o->bytes, q->p, q->bytes)) return true;
  }
  return false;
}

RowArgs row_args(const void* a, const void* w, int64_t w_stride, void* out, const void* gu,
                 const ExpertRows& rows, int64_t K, int64_t N, int act) {
  RowArgs p = {};
  p.a = static_cast<const char*>(a);
  p.w = static_cast<const char*>(w);
  p.w_stride = w_stride;
  p.out = static_cast<char*>(out);
  p.gu = static_cast<char*>(const_cast<void*>(gu));
  p.rows = rows;
  p.K = static_cast<int>(K);
  p.N = static_cast<int>(N);
  p.act = act;
  return p;
}

}  // namespace
}  // namespace moe

extern "C" int moe_expert_ffn(const void* x, int64_t R, int64_t H, int64_t F, int E,
                              const int32_t* expert_first, const int32_t* expert_count,
                              const void* w_in, const void* w_down, int dtype, int act, void* gu,
                              void* a, void* y, int32_t* d_err, void* stream) {
  if (const int st = moe::ffn_check(R, H, F, E, dtype, act)) return st;
  if (R == 0) return MOE_OK;
  if (x == nullptr || expert_first == nullptr || expert_count == nullptr || w_in == nullptr ||
      w_down == nullptr || a == nullptr || y == nullptr)
    return MOE_ERR_NULL;
  if (!moe::aligned16({x, w_in, w_down, gu, a, y})) return MOE_ERR_ALIGN;
  const int64_t es = dtype == MOE_BF16 ? 2 : 4;
  const int64_t w = E * H * F * es;
  if (moe::any_overlap({{gu, R * 2 * F * es}, {a, R * F * es}, {y, R * H * es}},
                       {{x, R * H * es}, {w_in, 2 * w}, {w_down, w}, {expert_first, E * int64_t{4}},
                        {expert_count, E * int64_t{4}}}))
    return MOE_ERR_SHAPE;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const moe::ExpertRows rows = {expert_first, expert_count, d_err, E, static_cast<int>(R)};
  if (const int st = moe::row_product<moe::kUp>(
          moe::row_args(x, w_in, 2 * F * H * es, a, gu, rows, H, F, act), dtype, s))
    return st;
  return moe::row_product<moe::kDown>(
      moe::row_args(a, w_down, H * F * es, y, nullptr, rows, F, H, act), dtype, s);
}

extern "C" int moe_expert_ffn_backward_workspace_size(int64_t R, int64_t H, int64_t F, int E,
                                                      int dtype, size_t* ws_bytes) {
  if (ws_bytes == nullptr) return MOE_ERR_NULL;
  if (const int st = moe::ffn_check(R, H, F, E, dtype, MOE_ACT_SILU)) return st;
  const moe::WeightPlan in = moe::weight_plan(R, E, 2 * F, H, dtype);
  const moe::WeightPlan down = moe::weight_plan(R, E, H, F, dtype);
  *ws_bytes = static_cast<size_t>(moe::backward_space(R, F, dtype, in, down).all);
  return MOE_OK;
}

extern "C" int moe_expert_ffn_backward(const void* dy, const void* x, int64_t R, int64_t H,
                                       int64_t F, int E, const int32_t* expert_first,
                                       const int32_t* expert_count, const void* w_in,
                                       const void* w_down, const void* gu, const void* a,
                                       int dtype, int act, void* dx, void* dw_in, void* dw_down,
                                       int32_t* d_err, void* ws, size_t ws_bytes, void* stream) {
  if (const int st = moe::ffn_check(R, H, F, E, dtype, act)) return st;
  if (expert_first == nullptr || expert_count == nullptr || dw_in == nullptr || dw_down == nullptr)
    return MOE_ERR_NULL;
  if (R > 0 && (dy == nullptr || x == nullptr || w_in == nullptr || w_down == nullptr ||
                gu == nullptr || a == nullptr || dx == nullptr || ws == nullptr))
    return MOE_ERR_NULL;
  if (!moe::aligned16({dy, x, w_in, w_down, gu, a, dx, dw_in, dw_down, ws})) return MOE_ERR_ALIGN;
  const int64_t es = dtype == MOE_BF16 ? 2 : 4;
  const int64_t w = E * H * F * es, dgu = R * 2 * F * es;
  const moe::WeightPlan plan_in = moe::weight_plan(R, E, 2 * F, H, dtype);
  const moe::WeightPlan plan_down = moe::weight_plan(R, E, H, F, dtype);
  const moe::BackwardSpace space = moe::backward_space(R, F, dtype, plan_in, plan_down);
  if (ws_bytes < static_cast<size_t>(space.all)) return MOE_ERR_WORKSPACE;
  if (moe::any_overlap({{dx, R * H * es}, {dw_in, 2 * w}, {dw_down, w}, {ws, space.all}},
                       {{dy, R * H * es}, {x, R * H * es}, {w_in, 2 * w}, {w_down, w}, {gu, dgu},
                        {a, dgu / 2}, {expert_first, E * int64_t{4}}, {expert_count, E * int64_t{4}}}))
    return MOE_ERR_SHAPE;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const moe::ExpertRows rows = {expert_first, expert_count, d_err, E, static_cast<int>(R)};
  if (R > 0)
    if (const int st = moe::row_product<moe::kActGrad>(
            moe::row_args(dy, w_down, H * F * es, ws, gu, rows, H, F, act), dtype, s))
      return st;
  moe::WeightArgs in = {};
  in.rows = rows;
  in.partial = reinterpret_cast<float*>(static_cast<char*>(ws) + space.in);
  in.p = static_cast<const char*>(ws);
  in.q = static_cast<const char*>(x);
  in.out = static_cast<char*>(dw_in);
  in.M = static_cast<int>(2 * F);
  in.N = static_cast<int>(H);
  moe::WeightArgs down = in;
  down.partial = reinterpret_cast<float*>(static_cast<char*>(ws) + space.down);
  down.p = static_cast<const char*>(dy);
  down.q = static_cast<const char*>(a);
  down.out = static_cast<char*>(dw_down);
  down.M = static_cast<int>(H);
  down.N = static_cast<int>(F);
  return moe::gradients(moe::row_args(ws, w_in, 2 * F * H * es, dx, nullptr, rows, 2 * F, H, act), in, down,
                        plan_in, plan_down, dtype, s);
}
