// Grouped matrix products on MFMA tiles (bf16 in, fp32 accumulation), the
// machinery of the experts' feed-forward block (ffn.hip).  Measured on MI355X,
// 64 experts of 4096 x 2048 with 1024 rows each on average: up 2.2 ms (1.0
// PFLOP/s), down 1.13 (0.97), activation gradient 1.23 (0.89), dx 2.0 (1.1),
// dWin 2.34 (0.94), dWdown 1.13 (0.97).  MFMAs are issued in 51 to 66% of a CU's
// cycles: a step of 64 k of up takes 1.5 us, its matrix work 1.0.  The rest is
// waiting and not the rate of the way from L2 into LDS: up and down, with two
// stages of 64 k whose loads all go out in the first of a step's two memory
// turns, have their waves wait (loads and barriers) 36% of the time and take 0.13
// cache lines a CU and cycle from L2; dx, with four stages of 32 k, waits 25% and
// takes 0.22.
//
// A block of WM x WN waves computes a BM x BN tile of C = A B, held as 16x16
// accumulators: MF row fragments (every WM-th one of the tile, so that a tile
// with few rows has all its waves share them) by NF column fragments a wave.
// K advances in steps of BK, 64 or 32.  Each step's operand tiles go from
// memory straight to LDS (16-byte buffer loads, no registers), into a ring of
// STAGES.
//
// 64 k are 128 bytes, a whole cache line of an operand whose k is contiguous:
// with 32 every line is asked for twice, and the L2's request rate counts.
// Steps of 32 k fill a finer ring, which gives the loads more time.
//
// An operand tile lies in LDS in the order of its memory:
//  - K contiguous (rows of activations, weights as [out][in]): [row][BK],
//    rows whose 16-byte chunks are permuted by the row, so that
//    the lanes that a fragment read serves together fall on all 64 banks;
//  - K major (weights read along their other axis; both operands of a weight
//    gradient): [BK][columns], read back through the LDS transpose reads
//    (ds_read_b64_tr_b16), chunks permuted by the row's low bits for the same
//    reason.
// The permutation is done by choosing which chunk a lane fetches: the LDS
// side of such a load is always linear in the lane.
//
// Out-of-range rows, columns and k are lanes whose offset lies outside the
// buffer descriptor: the load returns zero, so nothing past an expert's rows
// or the matrix edges is read and every K tail multiplies zeros by zeros.
#pragma once

#include "rowio.hpp"

namespace moe {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kOut = 0x7fffff00;  // a byte offset outside every descriptor

typedef __attribute__((address_space(3))) char* lds_ptr;
typedef int i32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ uint32_t lds_address(const char* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_ptr)const_cast<char*>(p)));
}

// A buffer descriptor for `bytes` bytes from p (fewer than kOut).
__device__ __forceinline__ i32x4 buffer_of(const char* p, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(p);
  i32x4 r;
  r[0] = __builtin_amdgcn_readfirstlane(static_cast<int>(a));
  r[1] = __builtin_amdgcn_readfirstlane(static_cast<int>((a >> 32) & 0xFFFF));
  r[2] = __builtin_amdgcn_readfirstlane(static_cast<int>(bytes));
  r[3] = 0x00020000;
  return r;
}

// Sixteen bytes a lane from buffer offset voff to LDS at lds + 16 * lane
// (lds uniform).  Written as an instruction because the compiler, which
// cannot tell the stages of the LDS ring apart, would wait for every load in
// flight before each LDS read; there is no output register, and the loops
// below wait for these loads themselves (stage_barrier).  M0, the
// instruction's LDS base, is set right before it; nothing else in these
// kernels takes a value through M0.
__device__ __forceinline__ void to_lds(i32x4 buffer, uint32_t lds, int voff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               ::"s"(lds), "v"(voff), "s"(buffer) : "memory");
}

// The chunk permutation of a row: chunk c lies at c ^ contig_rot(row).  A
// 16-byte LDS read serves 16 lanes at a time, rows 0-3 and 12-15 of one lane
// group with rows 4-11 of the next (whose chunk is the neighbour, c ^ 1).
// With two 128-byte rows to a 256-byte bank row and row / 2 as the
// permutation, or four 64-byte rows and row / 4 mapped to 0, 2, 3, 1, these
// are 16 different 16-byte columns (SQ_LDS_BANK_CONFLICT is 0).
template <int BK>
__device__ __forceinline__ int contig_rot(int row) {
  if constexpr (BK == 64) return (row >> 1) & 7;
  const int q = (row >> 2) & 3;
  return (((q ^ (q >> 1)) & 1) << 1) | (q >> 1);
}

// Which rotation row k of a K-major tile has: bits 0, 1 and 3 of k, on pairs
// of 16-byte chunks (a transpose read takes 32-byte pieces of 16 rows: k =
// 8 g + 4 j + r for its four lane groups g and rows r).
__device__ __forceinline__ int major_rot(int k) { return 2 * ((k & 3) | ((k >> 1) & 4)); }

// Loads a [ROWS][BK] tile of an operand whose k is contiguous.
template <int ROWS, int THREADS, int BK>
struct ContigTile {
  static constexpr int kChunks = BK / 8;
  static constexpr int kLoads = ROWS * kChunks / THREADS;
  static constexpr int kBytes = ROWS * BK * 2;
  int voff[kLoads];
  int chunk;  // first k of this lane's chunk

  // row_of(r): the operand row of tile row r, or -1.
  template <class RowOf>
  __device__ __forceinline__ void init(int64_t ld, RowOf row_of) {
    const int tid = threadIdx.x;
    chunk = ((tid % kChunks) ^ contig_rot<BK>(tid / kChunks)) * 8;  // the same for every load: rows 16 n apart
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int row = row_of(i * (THREADS / kChunks) + tid / kChunks);
      voff[i] = row < 0 ? kOut : static_cast<int>(row * ld * 2 + chunk * 2);
    }
  }
  // base: the operand's first row, `bytes` its extent; k0: a step's first k
  // of K.
  struct Step {
    i32x4 buffer;
    bool in;
  };
  __device__ __forceinline__ Step step(const char* base, uint32_t bytes, int k0, int K) const {
    return {buffer_of(base + static_cast<int64_t>(k0) * 2, bytes), k0 + chunk < K};
  }
  __device__ __forceinline__ void load(const Step& s, int i, uint32_t lds) const {
    to_lds(s.buffer, lds + (i * THREADS + wave_id() * kWave) * 16, s.in ? voff[i] : kOut);
  }
};

// Loads a [BK][COLS] tile of an operand whose columns are contiguous.
template <int COLS, int THREADS, int BK>
struct MajorTile {
  static constexpr int kChunks = COLS / 8;
  static constexpr int kLoads = BK * kChunks / THREADS;
  static constexpr int kBytes = COLS * BK * 2;
  int voff[kLoads];
  int row0;

  // cols: valid columns of the tile.
  __device__ __forceinline__ void init(int64_t ld, int cols) {
    const int tid = threadIdx.x;
    row0 = tid / kChunks;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int k = i * (THREADS / kChunks) + row0;
      const int c = ((tid % kChunks) ^ (major_rot(k) & (kChunks - 1))) * 8;
      voff[i] = c < cols ? static_cast<int>(k * ld * 2 + c * 2) : kOut;
    }
  }
  struct Step {
    i32x4 buffer;
    int rows;
  };
  // base: the tile's first column at k = 0.
  __device__ __forceinline__ Step step(const char* base, int64_t ld, int k0, int K) const {
    return {buffer_of(base + static_cast<int64_t>(k0) * ld * 2, static_cast<uint32_t>(BK * ld * 2)), K - k0};
  }
  __device__ __forceinline__ void load(const Step& s, int i, uint32_t lds) const {
    to_lds(s.buffer, lds + (i * THREADS + wave_id() * kWave) * 16,
           i * (THREADS / kChunks) + row0 < s.rows ? voff[i] : kOut);
  }
};

// Fragments of half h (32 k) of a [ROWS][BK] tile: lane l holds k = 32 h +
// 8 (l / 16) .. + 7 of row l % 16.
template <int BK>
struct ContigRead {
  int off[BK / 32];
  __device__ __forceinline__ void init(int row0) {
    const int l = lane_id();
#pragma unroll
    for (int h = 0; h < BK / 32; ++h)
      off[h] = (row0 + (l & 15)) * BK * 2 + ((h * 4 + (l >> 4)) ^ contig_rot<BK>(l & 15)) * 16;
  }
  // The fragment of rows row0 + 16 f ...
  __device__ __forceinline__ bf16x8 get(const char* lds, int f, int h) const {
    return *reinterpret_cast<const bf16x8*>(lds + off[h] + f * 16 * BK * 2);
  }
};

// Which columns a fragment's 16 are.  A lane's accumulator holds four of them
// (4 g .. + 3 for lane group g = lane / 16).  Column fragments go in pairs
// whose accumulators together are eight consecutive columns, one 16-byte
// store (or load) of bf16: column 8 g + 4 b + e of the pair's 32 is number
// 4 g + e of its fragment b.  Stored one fragment at a time, in 8 bytes, a
// tile's results took as long as a fifth of its products.
__device__ __forceinline__ int paired_column(int n) {  // n = 16 fragment + number
  return (n >> 5) * 32 + ((n >> 2) & 3) * 8 + ((n >> 4) & 1) * 4 + (n & 3);
}

// The same fragments out of a [BK][COLS] tile: two transpose reads of four
// k each; F fragments of 16 columns, STEP columns apart, from column col0.
// PAIRED: fragments 2 p and 2 p + 1 are the pairs above, but in lane groups 2
// and 3 the two have changed places (accumulators too): a read then takes 8
// bytes from each of 64 different banks, which two halves of the same side
// would not.
template <int COLS, int F, int STEP, bool PAIRED>
struct MajorRead {
  int off[F];
  __device__ __forceinline__ void init(int col0) {
    const int l = lane_id();
    const int k = (l >> 4) * 8 + ((l & 15) >> 2);
    const int piece = l & 3;  // four columns of the fragment
#pragma unroll
    for (int f = 0; f < F; ++f) {
      const int col = PAIRED ? col0 + (f >> 1) * 32 + piece * 8 + ((f & 1) ^ (piece >> 1)) * 4
                             : col0 + f * STEP + piece * 4;
      off[f] = k * COLS * 2 + ((col / 8) ^ (major_rot(k) & (COLS / 8 - 1))) * 16 + (col & 4) * 2;
    }
  }
  __device__ __forceinline__ bf16x8 get(const char* lds, int f, int h) const {
    typedef __attribute__((address_space(3))) s16x4* tr_ptr;
    char* p = const_cast<char*>(lds) + off[f] + h * 32 * COLS * 2;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((tr_ptr)p);
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((tr_ptr)(p + 4 * COLS * 2));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  }
};

// Waits until at most OUTSTANDING of the wave's loads and stores are.
template <int OUTSTANDING>
__device__ __forceinline__ void wait_loads() {
  constexpr int N = OUTSTANDING < 63 ? OUTSTANDING : 63;  // the counter's most
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
  __builtin_amdgcn_sched_barrier(0);
}

// Ends a turn: the wave's LDS reads are done, and every wave is here.
__device__ __forceinline__ void turn() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (3 << 14));  // lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

template <int MF, int NF>
struct Frags {
  bf16x8 a[MF];
  bf16x8 b[NF];
};

// A block's products, one tile after another.
//
// The two waves that share a SIMD (w and w + 4) take turns: while one
// multiplies 32 k (a half of a step), the other reads its next fragments from
// LDS and issues loads, and a barrier ends each turn.  The matrix pipe then
// always has a wave that does nothing else; with reads and loads dealt out
// between the MFMAs of both, a wave whose load waited for the texture pipe
// held up its own MFMAs and, in step with it, its neighbour's.
//
// A step's stage is free when both groups have read its second half.  The
// loads of step t - 1 + STAGES go out into the stage of step t - 1 in the
// memory turns of step t.
//
// Before a tile is stored, the loads of the next one's first STAGES steps are
// under way, so that a block never waits for memory with nothing in flight
// but its stores.  They are older than the tile's stores, so the next tile's first
// waits leave as many operations outstanding as there are stores.
//
// T, the kernel's tiles:
//   LOADS                  loads a wave issues a step
//   STORES                 stores a wave issues in store(), at least: no
//                          branch may leave one out
//   Work                   a tile; .steps (may be 0), .used: the wave's row
//                          fragments that hold rows (the rest are skipped)
//   bool tile(int i, Work&)  the block's i-th tile
//   void aim(const Work&)  prepares to load it
//   void begin(int step)   prepares the loads of a step of it (past its last:
//                          loads of nothing)
//   void load(i, stage)    issues load i of a step
//   read_a(i, stage, half, f), read_b(j, stage, half, f)   fetch one fragment
//   store(const Work&, acc)
template <int STAGES, int HALVES, int MF, int NF, class T>
__device__ __forceinline__ void tile_loop(T& tiles) {
  static_assert(STAGES >= 2, "a stage in use and one in flight");
  constexpr int LOADS = T::LOADS;
  constexpr int kSkip = MF / 2;  // row fragments that are skipped together
  constexpr int kLate = T::STORES;  // operations younger than a tile's first loads
  typename T::Work w;
  if (!tiles.tile(0, w)) return;
  auto prologue = [&] {
#pragma unroll
    for (int s = 0; s < STAGES; ++s) {
      tiles.begin(s);
#pragma unroll
      for (int i = 0; i < LOADS; ++i) tiles.load(i, s);
    }
  };
  if (w.steps > 0) {
    tiles.aim(w);
    prologue();
  }
  for (int tile = 0;;) {
    f32x4 acc[NF][MF];
#pragma unroll
    for (int j = 0; j < NF; ++j)
#pragma unroll
      for (int i = 0; i < MF; ++i) acc[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (w.steps > 0) {
      Frags<MF, NF> f;
      const bool leads = wave_id() < 4;
      auto multiply = [&](int i) {
#pragma unroll
        for (int j = 0; j < NF; ++j)
          acc[j][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f.b[j], f.a[i], acc[j][i], 0, 0, 0);
      };
      // The wave's own loads of the step that is read next have arrived.
      auto arrived = [&](bool late) {
        if (late)
          wait_loads<(STAGES - 2) * LOADS + kLate>();
        else
          wait_loads<(STAGES - 2) * LOADS>();
      };
      if (tile == 0)
        wait_loads<(STAGES - 1) * LOADS>();
      else
        wait_loads<(STAGES - 1) * LOADS + kLate>();
      turn();
      if (!leads) turn();
      for (int s = 0; s < w.steps; s += STAGES) {
#pragma unroll
        for (int u = 0; u < STAGES; ++u) {
          if (s + u < w.steps) {
            const bool late = tile > 0 && s == 0 && u < STAGES - 1;
#pragma unroll
            for (int h = 0; h < HALVES; ++h) {
              // Memory turn.
#pragma unroll
              for (int j = 0; j < NF; ++j) tiles.read_b(j, u, h, f.b[j]);
#pragma unroll
              for (int i = 0; i < MF; ++i) tiles.read_a(i, u, h, f.a[i]);
              if (s + u > 0) {
                // Two stages: all in the first half, to arrive in time.
                constexpr int kFirst = STAGES > 2 && HALVES > 1 ? LOADS / 2 : LOADS;
                if (h == 0) tiles.begin(s + u - 1 + STAGES);
#pragma unroll
                for (int q = h == 0 ? 0 : kFirst; q < (h == 0 ? kFirst : LOADS); ++q)
                  tiles.load(q, (u + STAGES - 1) % STAGES);
              }
              if (h == HALVES - 1 && !leads) arrived(late);
              turn();
              // Matrix turn.
              __builtin_amdgcn_s_setprio(1);
#pragma unroll
              for (int i = 0; i < MF; i += kSkip) {
                if (i < w.used) {
#pragma unroll
                  for (int q = i; q < i + kSkip; ++q) multiply(q);
                }
              }
              __builtin_amdgcn_s_setprio(0);
              if (h == HALVES - 1 && leads) arrived(late);
              turn();
            }
          }
        }
      }
      if (leads) turn();
      // Loads past the last step fetch nothing but still write zeros to LDS:
      // they end before the stages are filled again, and before the block does.
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    }
    typename T::Work next;
    const bool more = tiles.tile(++tile, next);
    if (more && next.steps > 0) {
      tiles.aim(next);
      prologue();
    }
    tiles.store(w, acc);
    if (!more) break;
    w = next;
  }
}

}  // namespace moe
