// The combine that closes a layer, and its backward pass.
//
//   b_t = sum_q a(row_q) z[row_q]          the block's output (combine.hip)
//   y_t = s x_t + gate_t (b_t rho_t) w_post,  rho = 1 / sqrt(mean(b^2) + eps)
//   h_t = (y_t sigma_t) w_next,             sigma = 1 / sqrt(mean(y^2) + eps)
//
// One pass: a token's rows, its residual row and both norms' weights meet in
// registers, so b never exists in memory and y is not read back for the
// next block's norm.  HBM-bound: (rows + x + y + h) row bytes a token.
//
// Backward, with D = dL/dy + the second norm's gradient:
//   D    = dy + sigma dh w_next - y sigma^3 <dh w_next, y> / H
//   dx   = s D
//   v    = D w_post;  P = <v, b>
//   db   = gate rho (v - b rho^2 P / H),  dz[row_q] = a_q db
//   dgate = rho P
//   da_q = <db, z_q> = gate rho^3 (eps S_q + sum_p a_p (S_q B_p - S_p B_q) / H)
//          with S_q = <v, z_q>, B_q = <b, z_q> (rho^-2 = <b, b>/H + eps, and
//          <b, b> = sum_p a_p B_p, P = sum_p a_p S_p): the term p = q drops
//          out, so a token with one row, whose weight the norm makes almost
//          irrelevant, gets its eps-sized gradient and not the difference of
//          two large sums.  Formed term by term in 64 bits, where products of
//          two fp32 numbers are exact and the term p = q is 0, and rounded
//          after the factor gate rho^3: the sum alone grows with the cube of z
//          and leaves the range of fp32 for |z| from 10^12 on
//   dw_post = sum_t gate D b rho,  dw_next = sum_t dh y sigma
// The norms' statistics are formed again from b and y (the rows are read
// anyway).  The token's rows of z are held in registers as loaded, so the two
// passes over them (b, then the dot products) cost one read (two where k > 4
// and rows are over 16 KiB); a block walks tokens and keeps the weight
// gradients in registers or LDS, and its sums go to the workspace once, where
// a second kernel adds them in a fixed order.
//
// Both kernels are a chain a token: row ids, rows, a sum over the row, and
// stores.  So they load one token ahead: the next token's row ids come with
// this one's rows, and its rows are asked for as soon as this token's are
// used up, before the sums and stores that follow.  Rows are read and written
// through buffer descriptors of one row: a missing row is a descriptor of no
// bytes, which reads zeros and drops stores, and so are the groups past a
// row's end, so the loads and stores have no branches around them and stay in
// flight together.
//
// All sums are fp32 (the few numbers of da_q: double); values are rounded
// once, when stored.
//
// Measured on MI355X, bf16, all inputs and outputs given.  Forward: 65536
// tokens, rows of 4096, two a token: 455 us for 2.62 GB, 5.8 TB/s (a copy
// reaches 6.6); 32768 tokens, rows of 7168, eight a token: 915 us, 5.6 TB/s.
// Backward: the same 65536 tokens 843 us for 4.3 GB, 5.1 TB/s; 16384 tokens,
// rows of 7168, eight a token 920 us, 5.0 TB/s.  fp32, 32768 tokens, rows of
// 4096, two a token: 455 us forward, 5.9 TB/s, 797 backward, 5.4 TB/s.  Vector
// instructions fill a good half of the backward's time, which is why its sums
// go four at a time and its weights through buffers.
//
// Rows that need two groups a thread or more do not fit the registers: the
// compiler spills 16 (bf16, k <= 2), 54 (bf16, k <= 4) or 22 (fp32, k <= 4) of
// the 128 that 1024 threads have (rows over 16 KiB), and 19 of the 256 that 512
// have (bf16, k > 4, rows over 8 KiB; 8 over 16 KiB); of the forward 26 (bf16,
// k > 4, rows over 16 KiB).  16384 tokens, bf16 rows of 16384, backward: two a
// token 867 us, 5.0 TB/s, but four a token 2078 us, 3.1 TB/s; 8192 tokens, eight
// a token 656 us forward, 4.5 TB/s, 1100 backward, 4.9 TB/s.
#include <math.h>

#include "rowio.hpp"

namespace moe {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

struct NormArgs {
  const u32x4* z;
  const u32x4* x;
  const u32x4* y;   // backward
  const u32x4* dy;  // backward, may be null
  const u32x4* dh;  // backward, may be null
  u32x4* y_out;     // may be null
  u32x4* h_out;     // may be null
  u32x4* dx;
  u32x4* dz;
  const int32_t* rows;
  const float* weight;
  const float* gate;
  const float* w_post;
  const float* w_next;
  float* d_weight;  // may be null
  float* d_gate;    // may be null
  float* partial;   // [blocks][2][H]: dw_post, dw_next
  const int32_t* n_valid;
  int32_t* d_err;
  int64_t z_rows;
  int T, H, groups, k;
  float scale, eps;
};

constexpr int kNormWaves = 16;                     // most waves of a block
constexpr int kNormThreads = kNormWaves * kWave;   // 1024
constexpr int64_t kNormCus = 256;
constexpr int kMaxSums = (2 * MOE_MAX_K + 2 + 3) / 4 * 4;  // written four at a time
static_assert(kMaxSums <= 32, "two half waves share the sums of a block");

// Sums of NV values over the threads that share a token: a wave, or the
// block (one barrier; `buf` alternates between two LDS buffers, so that a
// buffer is written again only after a barrier that follows its readers).
// After the barrier lane i of every wave adds value i % 32 of the even or odd
// waves, so a thread reads at most eight words whatever NV is.
template <int NV, bool WAVE>
__device__ __forceinline__ void token_sums(float (&v)[NV], float (*buf)[kMaxSums]) {
  constexpr int kQuads = (NV + 3) / 4;
  float part[kQuads];
#pragma unroll
  for (int r = 0; r < kQuads; ++r)
    part[r] = NV == 1 ? wave_sum_f(v[0]) : wave_sum_4(
        v[4 * r], 4 * r + 1 < NV ? v[4 * r + 1] : 0.f, 4 * r + 2 < NV ? v[4 * r + 2] : 0.f,
        4 * r + 3 < NV ? v[4 * r + 3] : 0.f);
  if constexpr (WAVE) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      v[i] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(part[i / 4]), i % 4 * 16));
  } else {
    const int waves = blockDim.x / kWave;
    if ((lane_id() & 15) == 0) {
#pragma unroll
      for (int r = 0; r < kQuads; ++r) buf[wave_id()][4 * r + (lane_id() >> 4)] = part[r];
    }
    __syncthreads();
    const int i = lane_id() & 31;
    float s = 0.f;
    if (i < NV)
      for (int w = lane_id() >> 5; w < waves; w += 2) s += buf[w][i];
    s += __shfl_xor(s, 32, kWave);
#pragma unroll
    for (int j = 0; j < NV; ++j)
      v[j] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(s), j));
  }
}

// A token's row ids and weights: loaded a slot a lane, then made uniform.
struct TokenRows {
  int id;
  float w;

  // Issues the load of token t's row ids (none from T on).
  __device__ __forceinline__ void ask(const NormArgs& p, int64_t t, int T) {
    id = lane_id() < p.k && t < T ? p.rows[t * p.k + lane_id()] : -1;
  }
  // Checks the ids and issues the load of their weights.
  __device__ __forceinline__ void check(const NormArgs& p, bool reports) {
    if (id >= p.z_rows) {
      if (reports) report(p.d_err, MOE_DERR_ROW_RANGE);
      id = -1;
    }
    w = id < 0 ? 0.f : (p.weight != nullptr ? p.weight[id] : 1.f);
  }
  template <int K>
  __device__ __forceinline__ void ids(int (&rid)[K]) const {
#pragma unroll
    for (int q = 0; q < K; ++q) rid[q] = __builtin_amdgcn_readlane(id, q);
  }
  template <int K>
  __device__ __forceinline__ void weights(float (&a)[K]) const {
#pragma unroll
    for (int q = 0; q < K; ++q)
      a[q] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(w), q));
  }
};

// One row as a buffer of its own; absent rows have no bytes.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_buffer(const u32x4* base, int64_t row, int groups,
                                                             bool present) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<u32x4*>(base) + row * groups, 0,
                                           present ? groups * 16 : 0, 0x00020000);
}

constexpr int kNontemporal = 2;  // the cache policy's nt bit

__device__ __forceinline__ u32x4 row_load(__amdgpu_buffer_rsrc_t r, int g) {
  return __builtin_amdgcn_raw_buffer_load_b128(r, g * 16, 0, kNontemporal);
}

template <bool BF16>
struct Elems {
  static constexpr int value = BF16 ? 8 : 4;  // elements of a 16-byte group
};

template <bool BF16, int EPL>
__device__ __forceinline__ void unpack(u32x4 v, float (&f)[EPL]) {
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    if constexpr (BF16)
      f[i] = (i & 1) ? bf16_hi(v[i / 2]) : bf16_lo(v[i / 2]);
    else
      f[i] = __uint_as_float(v[i]);
  }
}

// Rounds and stores one group of a row.
template <bool BF16, int EPL>
__device__ __forceinline__ void row_store(__amdgpu_buffer_rsrc_t r, int g, const float (&f)[EPL]) {
  u32x4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF16) {
      typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
      const bf16x2 h = {static_cast<__bf16>(f[2 * i]), static_cast<__bf16>(f[2 * i + 1])};
      v[i] = __builtin_bit_cast(uint32_t, h);  // round to nearest even, one instruction
    } else {
      v[i] = __float_as_uint(f[i]);
    }
  }
  __builtin_amdgcn_raw_buffer_store_b128(v, r, g * 16, 0, kNontemporal);
}

// A norm's weights as a buffer: none, and groups past the row's end, read 0.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t weight_buffer(const float* w, int H) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(w), 0, w != nullptr ? H * 4 : 0, 0x00020000);
}

template <int EPL>
__device__ __forceinline__ void load_weights(__amdgpu_buffer_rsrc_t w, int g, float (&f)[EPL]) {
#pragma unroll
  for (int h = 0; h < EPL / 4; ++h) {
    const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(w, (g * (EPL / 4) + h) * 16, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[4 * h + i] = __uint_as_float(v[i]);
  }
}

template <bool BF16, int U, int K, bool WAVE>
__global__ __launch_bounds__(WAVE ? 256 : kNormThreads) void combine_norm_kernel(NormArgs p) {
  constexpr int EPL = Elems<BF16>::value;
  __shared__ float s_sum[2][kNormWaves][kMaxSums];
  const int T = p.n_valid != nullptr ? min(p.T, *p.n_valid) : p.T;
  const int lanes = WAVE ? kWave : static_cast<int>(blockDim.x);
  const int g0 = WAVE ? lane_id() : static_cast<int>(threadIdx.x);
  const int per = WAVE ? 256 / kWave : 1;
  const int first = static_cast<int>(blockIdx.x) * per + (WAVE ? wave_id() : 0);
  const int step = static_cast<int>(gridDim.x) * per;
  const float inv_h = 1.f / static_cast<float>(p.H);

  // Both weight vectors stay in registers while the block walks its tokens
  // (they are twice as wide as a bf16 row).
  float wp[U][EPL], wn[U][EPL];
  const auto post_weights = weight_buffer(p.w_post, p.H), next_weights = weight_buffer(p.w_next, p.H);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    load_weights<EPL>(post_weights, g0 + u * lanes, wp[u]);
    load_weights<EPL>(next_weights, g0 + u * lanes, wn[u]);
  }

  TokenRows ahead;
  int rid[K];
  float a[K];
  u32x4 xv[U], zv[K][U];
  auto load_x = [&](int64_t t) {
    const auto x = row_buffer(p.x, t, p.groups, t < T);
#pragma unroll
    for (int u = 0; u < U; ++u) xv[u] = row_load(x, g0 + u * lanes);
  };
  auto load_z = [&] {
    ahead.ids(rid);
#pragma unroll
    for (int q = 0; q < K; ++q) {
      const auto z = row_buffer(p.z, rid[q], p.groups, rid[q] >= 0);
#pragma unroll
      for (int u = 0; u < U; ++u) zv[q][u] = row_load(z, g0 + u * lanes);
    }
  };
  if (p.k > 0) {
    ahead.ask(p, first, T);
    ahead.check(p, g0 < kWave);
    load_z();
  }
  load_x(first);

  for (int64_t t = first; t < T; t += step) {
    const float gate = p.gate != nullptr
        ? __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(p.gate[t]))) : 1.f;
    float b[U][EPL];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < EPL; ++i) b[u][i] = 0.f;
    float post = 0.f;
    if (p.k > 0) {
      ahead.weights(a);
      ahead.ask(p, t + step, T);
#pragma unroll
      for (int q = 0; q < K; ++q) {
        if (rid[q] < 0) continue;  // no product with an absent row's weight of 0
#pragma unroll
        for (int u = 0; u < U; ++u) {
          float f[EPL];
          unpack<BF16, EPL>(zv[q][u], f);
#pragma unroll
          for (int i = 0; i < EPL; ++i) b[u][i] = __builtin_fmaf(a[q], f[i], b[u][i]);
        }
      }
      ahead.check(p, g0 < kWave);
      load_z();
      float ss[1] = {0.f};
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < EPL; ++i) ss[0] = __builtin_fmaf(b[u][i], b[u][i], ss[0]);
      token_sums<1, WAVE>(ss, s_sum[0]);
      post = gate * rsqrtf(__builtin_fmaf(ss[0], inv_h, p.eps));
    }
    const auto y = row_buffer(p.y_out, t, p.groups, p.y_out != nullptr);
    float yy[1] = {0.f};
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float f[EPL];
      unpack<BF16, EPL>(xv[u], f);
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        // (b * post) * w: a padded group's weights are 0
        b[u][i] = __builtin_fmaf(b[u][i] * post, wp[u][i], p.scale * f[i]);
        yy[0] = __builtin_fmaf(b[u][i], b[u][i], yy[0]);
      }
    }
    load_x(t + step);
#pragma unroll
    for (int u = 0; u < U; ++u) row_store<BF16, EPL>(y, g0 + u * lanes, b[u]);
    if (p.h_out != nullptr) {
      const auto h = row_buffer(p.h_out, t, p.groups, true);
      token_sums<1, WAVE>(yy, s_sum[1]);
      const float sigma = rsqrtf(__builtin_fmaf(yy[0], inv_h, p.eps));
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float f[EPL];
#pragma unroll
        for (int i = 0; i < EPL; ++i) f[i] = b[u][i] * sigma * wn[u][i];
        row_store<BF16, EPL>(h, g0 + u * lanes, f);
      }
    }
    // The next token's sum goes to a buffer that is still being read, unless
    // both buffers are in use and the other one's barrier lies between.
    if (!WAVE && !(p.k > 0 && p.h_out != nullptr)) __syncthreads();
  }
}

// HOLD: the token's rows of z stay in registers between the two passes over
// them (K * U 16-byte groups a lane, at most 64 registers); otherwise the
// second pass reads them again.
template <bool BF16, int U, int K, bool WAVE>
__global__ __launch_bounds__(WAVE ? 256 : K > 4 ? kNormThreads / 2 : kNormThreads) void combine_norm_bwd_kernel(NormArgs p) {
  constexpr int EPL = Elems<BF16>::value;
  constexpr bool HOLD = K * U <= 16;
  __shared__ float s_sum[2][kNormWaves][kMaxSums];
  const int T = p.n_valid != nullptr ? min(p.T, *p.n_valid) : p.T;
  const int lanes = WAVE ? kWave : static_cast<int>(blockDim.x);
  const int g0 = WAVE ? lane_id() : static_cast<int>(threadIdx.x);
  const int per = WAVE ? 256 / kWave : 1;
  const int first = static_cast<int>(blockIdx.x) * per + (WAVE ? wave_id() : 0);
  const int step = static_cast<int>(gridDim.x) * per;
  const float inv_h = 1.f / static_cast<float>(p.H);

  // Both weight gradients: registers, or for a block's wide rows a private
  // piece of LDS each (32 registers fewer than the row's own values need).
  extern __shared__ f32x4 s_dw[];
  constexpr int kQuads = EPL / 4;
  float dw_reg[2][WAVE ? U : 1][EPL];
  auto dw_slot = [&](int which, int u, int h) -> f32x4& {
    return s_dw[((which * U + u) * kQuads + h) * lanes + g0];
  };
#pragma unroll
  for (int which = 0; which < 2; ++which)
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if constexpr (WAVE) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) dw_reg[which][u][i] = 0.f;
      } else {
#pragma unroll
        for (int h = 0; h < kQuads; ++h) dw_slot(which, u, h) = f32x4{0.f, 0.f, 0.f, 0.f};
      }
    }
  // Adds x * y to gradient `which`.
  auto dw_add = [&](int which, int u, const float (&x)[EPL], const float (&y)[EPL]) {
    if constexpr (WAVE) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) dw_reg[which][u][i] = __builtin_fmaf(x[i], y[i], dw_reg[which][u][i]);
    } else {
#pragma unroll
      for (int h = 0; h < kQuads; ++h) {
        f32x4 w = dw_slot(which, u, h);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __builtin_fmaf(x[4 * h + i], y[4 * h + i], w[i]);
        dw_slot(which, u, h) = w;
      }
    }
  };

  TokenRows ahead;
  int rid[K];
  float a[K];
  u32x4 yv[U], hv[U], dv[U], zv[HOLD ? K : 1][HOLD ? U : 1];
  auto load_rows = [&](int64_t t) {
    const auto y = row_buffer(p.y, t, p.groups, t < T && p.dh != nullptr);
    const auto h = row_buffer(p.dh, t, p.groups, t < T && p.dh != nullptr);
    const auto d = row_buffer(p.dy, t, p.groups, t < T && p.dy != nullptr);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      yv[u] = row_load(y, g0 + u * lanes);
      hv[u] = row_load(h, g0 + u * lanes);
      dv[u] = row_load(d, g0 + u * lanes);
    }
  };
  auto load_z = [&](const int (&id)[K]) {
    if constexpr (HOLD) {
#pragma unroll
      for (int q = 0; q < K; ++q) {
        const auto z = row_buffer(p.z, id[q], p.groups, id[q] >= 0);
#pragma unroll
        for (int u = 0; u < U; ++u) zv[q][u] = row_load(z, g0 + u * lanes);
      }
    }
  };
  const auto post_weights = weight_buffer(p.w_post, p.H), next_weights = weight_buffer(p.w_next, p.H);
  load_rows(first);
  if (p.k > 0) {
    ahead.ask(p, first, T);
    ahead.check(p, g0 < kWave);
    ahead.ids(rid);
    load_z(rid);
  }

  for (int64_t t = first; t < T; t += step) {
    int mine = -1;  // this lane's row
    if (p.k > 0) {
      ahead.weights(a);
      mine = ahead.id;
      ahead.ask(p, t + step, T);
    }
    // One group of a row of z in fp32.
    auto z_group = [&](int q, int u, float (&f)[EPL]) {
      if constexpr (HOLD)
        unpack<BF16, EPL>(zv[q][u], f);
      else
        unpack<BF16, EPL>(row_load(row_buffer(p.z, rid[q], p.groups, rid[q] >= 0), g0 + u * lanes), f);
    };

    // D, the whole gradient at y.
    float d[U][EPL];
#pragma unroll
    for (int u = 0; u < U; ++u) unpack<BF16, EPL>(dv[u], d[u]);
    if (p.dh != nullptr) {
      float s[2] = {0.f, 0.f};
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float yf[EPL], hf[EPL], wn[EPL];
        unpack<BF16, EPL>(yv[u], yf);
        unpack<BF16, EPL>(hv[u], hf);
        load_weights<EPL>(next_weights, g0 + u * lanes, wn);
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          s[0] = __builtin_fmaf(yf[i], yf[i], s[0]);
          s[1] = __builtin_fmaf(hf[i] * wn[i], yf[i], s[1]);
        }
      }
      token_sums<2, WAVE>(s, s_sum[0]);
      const float sigma = rsqrtf(__builtin_fmaf(s[0], inv_h, p.eps));
      const float c = s[1] * sigma * sigma * sigma * inv_h;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float yf[EPL], hf[EPL], wn[EPL];
        unpack<BF16, EPL>(yv[u], yf);
        unpack<BF16, EPL>(hv[u], hf);
        load_weights<EPL>(next_weights, g0 + u * lanes, wn);
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          d[u][i] = __builtin_fmaf(hf[i] * wn[i], sigma, __builtin_fmaf(-c, yf[i], d[u][i]));
          yf[i] *= sigma;
        }
        dw_add(1, u, hf, yf);
      }
    }
    const auto dx = row_buffer(p.dx, t, p.groups, true);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float f[EPL];
#pragma unroll
      for (int i = 0; i < EPL; ++i) f[i] = p.scale * d[u][i];
      row_store<BF16, EPL>(dx, g0 + u * lanes, f);
    }
    load_rows(t + step);
    if (p.k == 0) {
      if (g0 == 0 && p.d_gate != nullptr) p.d_gate[t] = 0.f;
      if (!WAVE && p.dh != nullptr) __syncthreads();  // s_sum[0]
      continue;
    }

    // b, then <b, b>, <v, b> and, for the weights, S_q and B_q.
    const float gate = p.gate != nullptr
        ? __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(p.gate[t]))) : 1.f;
    float b[U][EPL], v[U][EPL];
    float s[2 * K + 2];
#pragma unroll
    for (int i = 0; i < 2 * K + 2; ++i) s[i] = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float wp[EPL];
      load_weights<EPL>(post_weights, g0 + u * lanes, wp);
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        b[u][i] = 0.f;
        v[u][i] = d[u][i] * wp[i];
      }
#pragma unroll
      for (int q = 0; q < K; ++q) {
        float f[EPL];
        z_group(q, u, f);
#pragma unroll
        for (int i = 0; i < EPL; ++i) b[u][i] = __builtin_fmaf(a[q], f[i], b[u][i]);
      }
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        s[0] = __builtin_fmaf(b[u][i], b[u][i], s[0]);
        s[1] = __builtin_fmaf(v[u][i], b[u][i], s[1]);
      }
      if (p.d_weight != nullptr) {
#pragma unroll
        for (int q = 0; q < K; ++q) {
          // Unpacked again, not kept: K rows in fp32 would not fit.
          if constexpr (HOLD) asm volatile("" : "+v"(zv[q][u]));
          float f[EPL];
          z_group(q, u, f);
#pragma unroll
          for (int i = 0; i < EPL; ++i) {
            s[2 + q] = __builtin_fmaf(v[u][i], f[i], s[2 + q]);
            s[2 + K + q] = __builtin_fmaf(b[u][i], f[i], s[2 + K + q]);
          }
        }
      }
    }
    // This token's rows of z are used up: ask for the next one's (into the
    // same registers: not earlier).
    __builtin_amdgcn_sched_barrier(0);
    int next[K];
    ahead.check(p, g0 < kWave);
    ahead.ids(next);
    load_z(next);
    if (p.d_weight != nullptr) {
      token_sums<2 * K + 2, WAVE>(s, s_sum[1]);
    } else {
      float two[2] = {s[0], s[1]};
      token_sums<2, WAVE>(two, s_sum[1]);
      s[0] = two[0];
      s[1] = two[1];
    }
    const float rho = rsqrtf(__builtin_fmaf(s[0], inv_h, p.eps));
    const float c = s[1] * rho * rho * inv_h;
    const float gr = gate * rho;
    if (g0 == 0 && p.d_gate != nullptr) p.d_gate[t] = rho * s[1];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) d[u][i] *= gr;
      dw_add(0, u, d[u], b[u]);
#pragma unroll
      for (int i = 0; i < EPL; ++i) b[u][i] = __builtin_fmaf(-c, b[u][i], v[u][i]);  // db / (gate rho)
    }
    // The rows' weights: lane q has row q (a wave of the block).
    if (p.d_weight != nullptr && g0 < kWave) {
      float sq = 0.f, bq = 0.f;
      int listed = 0, before = 0;
#pragma unroll
      for (int o = 0; o < K; ++o) {
        sq = lane_id() == o ? s[2 + o] : sq;
        bq = lane_id() == o ? s[2 + K + o] : bq;
        const int same = rid[o] == mine ? 1 : 0;
        listed += same;
        before += lane_id() > o ? same : 0;
      }
      if (mine >= 0 && before == 0) {
        double cross = 0.0;
#pragma unroll
        for (int o = 0; o < K; ++o) {
          const double back = static_cast<double>(s[2 + o]) * bq;
          cross = __builtin_fma(a[o], __builtin_fma(sq, static_cast<double>(s[2 + K + o]), -back), cross);
        }
        const double r = rho, da = static_cast<double>(p.eps) * sq + cross * inv_h;
        p.d_weight[mine] = static_cast<float>(listed * static_cast<double>(gate) * r * r * r * da);
      }
    }
#pragma unroll
    for (int q = 0; q < K; ++q) {
      if (rid[q] < 0) continue;
      // A row listed twice by its token gets the gradient of both listings.
      int listed = 1;
      bool again = false;
#pragma unroll
      for (int o = 0; o < K; ++o) {
        if (o < q && rid[o] == rid[q]) again = true;
        if (o > q && rid[o] == rid[q]) ++listed;
      }
      if (again) continue;
      const float af = a[q] * gr * static_cast<float>(listed);
      const auto out = row_buffer(p.dz, rid[q], p.groups, true);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float o[EPL];
#pragma unroll
        for (int i = 0; i < EPL; ++i) o[i] = af * b[u][i];
        row_store<BF16, EPL>(out, g0 + u * lanes, o);
      }
    }
#pragma unroll
    for (int q = 0; q < K; ++q) rid[q] = next[q];
    if (!WAVE && p.dh == nullptr) __syncthreads();  // s_sum[1] is written again by the next token
  }

  // The block's share of both weight gradients (a wave per token: the four
  // waves' shares one after another through LDS).
  float* out = p.partial + static_cast<int64_t>(blockIdx.x) * 2 * p.H;
  if constexpr (WAVE) {
    __shared__ float s_w[2][kWave * U * EPL];
    for (int w = 0; w < 256 / kWave; ++w) {
      __syncthreads();
      if (wave_id() != w) continue;
#pragma unroll
      for (int which = 0; which < 2; ++which)
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int i = 0; i < EPL; ++i) {
            float& sum = s_w[which][(g0 + u * kWave) * EPL + i];
            sum = dw_reg[which][u][i] + (w > 0 ? sum : 0.f);
          }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < p.H; c += 256) {
      out[c] = s_w[0][c];
      out[p.H + c] = s_w[1][c];
    }
  } else {
#pragma unroll
    for (int which = 0; which < 2; ++which)
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int g = g0 + u * lanes;
        if (g < p.groups) {
#pragma unroll
          for (int h = 0; h < kQuads; ++h)
            *reinterpret_cast<f32x4*>(out + static_cast<int64_t>(which) * p.H + g * EPL + 4 * h) =
                dw_slot(which, u, h);
        }
      }
  }
}

// The blocks' shares added in a fixed order: 64 columns a block, 16 rows of
// shares at a time, then the 16 partial sums in LDS.
constexpr int kSumRows = 16;

__global__ __launch_bounds__(kWave* kSumRows) void norm_weight_sum_kernel(
    const float* __restrict__ partial, int n, int H, float* __restrict__ dw_post,
    float* __restrict__ dw_next) {
  __shared__ float s_part[kSumRows][kWave];
  const int lane = lane_id(), r = wave_id();
  const int c = static_cast<int>(blockIdx.x) * kWave + lane;
  float acc = 0.f;
  if (c < 2 * H) {
    const float* col = partial + c;
#pragma unroll 8
    for (int i = r; i < n; i += kSumRows) acc += col[static_cast<int64_t>(i) * 2 * H];
  }
  s_part[r][lane] = acc;
  __syncthreads();
  if (r != 0 || c >= 2 * H) return;
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < kSumRows; ++i) sum += s_part[i][lane];
  float* out = c < H ? dw_post : dw_next;
  if (out != nullptr) out[c < H ? c : c - H] = sum;
}

// A launch's shape: a wave a token up to 128 groups (2 KiB rows), else a
// block of up to 1024 threads a token with one group a thread, or two.  65536
// tokens, bf16 rows of 1024 (128 groups), six a token: 206 us forward and 439
// backward with a wave a token, 222 and 648 with a block of two waves.
struct NormShape {
  int unroll, threads, blocks;
  bool wave;
};

// Tokens a block of either mode takes at a time.
inline int64_t norm_tokens(int64_t groups) { return groups <= 2 * kWave ? 256 / kWave : 1; }

// Blocks of the forward.  A token each while there are at most eight blocks a
// CU; then two turns a block, up to 64 blocks a CU, so that a block's start
// (the norms' weights) is paid once for two turns or more and the last blocks
// end together.  65536 tokens, bf16, rows of 4096 and two a token: 499 us
// with eight blocks a CU that walk 32 tokens each, 470 with 64; 32768 tokens,
// rows of 7168, eight a token: 931 and 913, but 1137 with a token a block.
inline int forward_blocks(int64_t T, int64_t groups) {
  const int64_t per = norm_tokens(groups);
  const int64_t want = (T + per - 1) / per;
  const int64_t low = kNormCus * 8, high = kNormCus * 64;
  if (want <= low) return static_cast<int>(want);
  const int64_t two = (want + 1) / 2;
  return static_cast<int>(two < low ? low : two < high ? two : high);
}

// Blocks of the backward, which walk their tokens and add up the weight
// gradients on the way: two a CU, or as many as make 1024 threads.  Depends on
// T and the row alone, since the size of the workspace, a row of shares a
// block, does.  16384 tokens, bf16, rows of 2048 (blocks of 256 threads), two
// a token: 151 us with two blocks a CU, 120 with four, 128 with eight; rows of
// 1024 (a wave a token), 65536 tokens: 244 with one, 217 with two, 239 with
// four.
inline int backward_blocks(int64_t T, int64_t groups) {
  const int64_t per = norm_tokens(groups);
  const int64_t want = (T + per - 1) / per;
  const int64_t lanes = (groups + kWave - 1) / kWave * kWave;
  const int64_t fill = per == 1 ? kNormThreads / lanes : 0;
  const int64_t most = kNormCus * (fill > 2 ? fill : 2);
  return static_cast<int>(want < most ? (want > 0 ? want : 1) : most);
}

NormShape norm_shape(int blocks, int64_t groups, int most_threads) {
  NormShape s;
  s.wave = groups <= 2 * kWave;
  if (s.wave) {
    s.unroll = groups <= kWave ? 1 : 2;
    s.threads = 256;
  } else {
    s.unroll = 1;
    while (groups > static_cast<int64_t>(s.unroll) * most_threads) s.unroll *= 2;
    const int64_t lanes = (groups + s.unroll - 1) / s.unroll;
    s.threads = static_cast<int>((lanes + kWave - 1) / kWave * kWave);
  }
  s.blocks = blocks;
  return s;
}

// Most threads of the backward's blocks: more than four rows a token in
// registers need more than the 128 registers that 1024 threads have.
inline int bwd_threads(int k) { return k > 4 ? kNormThreads / 2 : kNormThreads; }

template <template <bool, int, int, bool> class Launch, bool BF16, int K>
void norm_launch_u(const NormShape& s, const NormArgs& p, hipStream_t st) {
  if (s.wave) {
    if (s.unroll == 1)
      Launch<BF16, 1, K, true>::go(s, p, st);
    else
      Launch<BF16, 2, K, true>::go(s, p, st);
  } else {
    if (s.unroll == 1)
      Launch<BF16, 1, K, false>::go(s, p, st);
    else if (s.unroll == 2)
      Launch<BF16, 2, K, false>::go(s, p, st);
    else if constexpr (Launch<BF16, 4, K, false>::kUsed)
      Launch<BF16, 4, K, false>::go(s, p, st);
  }
}

template <template <bool, int, int, bool> class Launch>
void norm_launch(const NormShape& s, const NormArgs& p, int dtype, hipStream_t st) {
  const bool bf = dtype == MOE_BF16;
  if (p.k <= 2)
    bf ? norm_launch_u<Launch, true, 2>(s, p, st) : norm_launch_u<Launch, false, 2>(s, p, st);
  else if (p.k <= 4)
    bf ? norm_launch_u<Launch, true, 4>(s, p, st) : norm_launch_u<Launch, false, 4>(s, p, st);
  else
    bf ? norm_launch_u<Launch, true, 8>(s, p, st) : norm_launch_u<Launch, false, 8>(s, p, st);
}

template <bool BF16, int U, int K, bool WAVE>
struct Forward {
  static constexpr bool kUsed = WAVE || U < 4;
  static void go(const NormShape& s, const NormArgs& p, hipStream_t st) {
    combine_norm_kernel<BF16, U, K, WAVE><<<s.blocks, s.threads, 0, st>>>(p);
  }
};

template <bool BF16, int U, int K, bool WAVE>
struct Backward {
  static constexpr bool kUsed = WAVE || U < 4 || K > 4;
  static void go(const NormShape& s, const NormArgs& p, hipStream_t st) {
    // Two fp32 gradients of the row, a private slot a thread and group.
    const unsigned lds = WAVE ? 0u : static_cast<unsigned>(2 * U * Elems<BF16>::value * sizeof(float) * s.threads);
    combine_norm_bwd_kernel<BF16, U, K, WAVE><<<s.blocks, s.threads, lds, st>>>(p);
  }
};

constexpr int64_t kMaxRowBytes = 2 * kNormThreads * 16;  // 32 KiB

int norm_check(int64_t T, int64_t H, int k, int64_t z_rows, int dtype, float scale, float eps) {
  if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_ERR_DTYPE;
  const int es = dtype == MOE_BF16 ? 2 : 4;
  if (T < 0 || T > INT32_MAX || H <= 0 || H * es > kMaxRowBytes || k < 0 || k > MOE_MAX_K ||
      z_rows < 0 || T * static_cast<int64_t>(k) >= (int64_t{1} << 31) || !(eps > 0.f) ||
      !isfinite(eps) || !isfinite(scale))
    return MOE_ERR_SHAPE;
  if (H * es % 16 != 0) return MOE_ERR_ALIGN;
  return MOE_OK;
}

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

}  // namespace
}  // namespace moe

extern "C" int moe_combine_norm(const void* z, int64_t z_rows, const int32_t* rows, int k,
                                const float* row_weight, const void* x, const float* gate,
                                const float* w_post, const float* w_next, float residual_scale,
                                float eps, int64_t T, int64_t H, int dtype, void* y, void* h,
                                const int32_t* n_valid, int32_t* d_err, void* stream) {
  if (const int st = moe::norm_check(T, H, k, z_rows, dtype, residual_scale, eps)) return st;
  if (T == 0) return MOE_OK;
  if (x == nullptr || (y == nullptr && h == nullptr) || (h != nullptr && w_next == nullptr) ||
      (k > 0 && (rows == nullptr || w_post == nullptr || (z == nullptr && z_rows > 0))))
    return MOE_ERR_NULL;
  if (!moe::aligned16(x) || !moe::aligned16(y) || !moe::aligned16(h) ||
      (k > 0 && (!moe::aligned16(z) || !moe::aligned16(w_post))) || !moe::aligned16(w_next))
    return MOE_ERR_ALIGN;
  const int64_t row = H * (dtype == MOE_BF16 ? 2 : 4);
  if (moe::overlap(y, T * row, x, T * row) || moe::overlap(h, T * row, x, T * row) ||
      moe::overlap(y, T * row, h, T * row) ||
      (k > 0 && (moe::overlap(y, T * row, z, z_rows * row) || moe::overlap(h, T * row, z, z_rows * row))))
    return MOE_ERR_SHAPE;
  moe::NormArgs p = {};
  p.z = static_cast<const moe::u32x4*>(z);
  p.x = static_cast<const moe::u32x4*>(x);
  p.y_out = static_cast<moe::u32x4*>(y);
  p.h_out = static_cast<moe::u32x4*>(h);
  p.rows = rows;
  p.weight = row_weight;
  p.gate = k > 0 ? gate : nullptr;
  p.w_post = k > 0 ? w_post : nullptr;
  p.w_next = h != nullptr ? w_next : nullptr;
  p.n_valid = n_valid;
  p.d_err = d_err;
  p.z_rows = z_rows;
  p.T = static_cast<int>(T);
  p.H = static_cast<int>(H);
  p.groups = static_cast<int>(row / 16);
  p.k = k;
  p.scale = residual_scale;
  p.eps = eps;
  const moe::NormShape s = moe::norm_shape(moe::forward_blocks(T, p.groups), p.groups, moe::kNormThreads);
  moe::norm_launch<moe::Forward>(s, p, dtype, static_cast<hipStream_t>(stream));
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}

extern "C" int moe_combine_norm_backward_workspace_size(int64_t T, int64_t H, int dtype,
                                                        size_t* ws_bytes) {
  if (ws_bytes == nullptr) return MOE_ERR_NULL;
  if (const int st = moe::norm_check(T, H, 0, 0, dtype, 1.f, 1.f)) return st;
  const int64_t groups = H * (dtype == MOE_BF16 ? 2 : 4) / 16;
  const int64_t blocks = moe::backward_blocks(T, groups);
  *ws_bytes = static_cast<size_t>(blocks) * 2 * H * sizeof(float);
  return MOE_OK;
}

extern "C" int moe_combine_norm_backward(
    const void* dy, const void* dh, const void* z, int64_t z_rows, const int32_t* rows, int k,
    const float* row_weight, const void* y, const float* gate, const float* w_post,
    const float* w_next, float residual_scale, float eps, int64_t T, int64_t H, int dtype,
    void* dx, void* dz, float* d_row_weight, float* d_gate, float* dw_post, float* dw_next,
    const int32_t* n_valid, int32_t* d_err, void* ws, size_t ws_bytes, void* stream) {
  if (const int st = moe::norm_check(T, H, k, z_rows, dtype, residual_scale, eps)) return st;
  if (ws == nullptr || (k > 0 && dw_post == nullptr) || (dh != nullptr && dw_next == nullptr))
    return MOE_ERR_NULL;
  if (T > 0 && ((dy == nullptr && dh == nullptr) || dx == nullptr ||
                (dh != nullptr && (y == nullptr || w_next == nullptr)) ||
                (k > 0 && (rows == nullptr || w_post == nullptr ||
                           (z_rows > 0 && (z == nullptr || dz == nullptr)) ||
                           (d_row_weight != nullptr && row_weight == nullptr)))))
    return MOE_ERR_NULL;
  if (!moe::aligned16(dy) || !moe::aligned16(dh) || !moe::aligned16(y) || !moe::aligned16(dx) ||
      !moe::aligned16(z) || !moe::aligned16(dz) || !moe::aligned16(w_post) ||
      !moe::aligned16(w_next) || !moe::aligned16(ws))
    return MOE_ERR_ALIGN;
  size_t need = 0;
  moe_combine_norm_backward_workspace_size(T, H, dtype, &need);
  if (ws_bytes < need) return MOE_ERR_WORKSPACE;
  const int64_t row = H * (dtype == MOE_BF16 ? 2 : 4);
  const int64_t space = static_cast<int64_t>(need);
  const void* in[3] = {dy, dh, dh != nullptr ? y : nullptr};
  for (const void* i : in)
    if (moe::overlap(dx, T * row, i, T * row) || moe::overlap(ws, space, i, T * row) ||
        (k > 0 && moe::overlap(dz, z_rows * row, i, T * row)))
      return MOE_ERR_SHAPE;
  if (moe::overlap(ws, space, dx, T * row)) return MOE_ERR_SHAPE;
  // A token's gate is read by all waves of its block, one of which writes d_gate.
  if (moe::overlap(d_gate, T * 4, gate, T * 4)) return MOE_ERR_SHAPE;
  if (k > 0 && (moe::overlap(dx, T * row, z, z_rows * row) ||
                moe::overlap(dx, T * row, dz, z_rows * row) ||
                moe::overlap(dz, z_rows * row, z, z_rows * row) ||
                moe::overlap(ws, space, z, z_rows * row) ||
                moe::overlap(ws, space, dz, z_rows * row)))
    return MOE_ERR_SHAPE;
  hipStream_t st = static_cast<hipStream_t>(stream);
  moe::NormArgs p = {};
  p.z = static_cast<const moe::u32x4*>(z);
  p.y = static_cast<const moe::u32x4*>(y);
  p.dy = static_cast<const moe::u32x4*>(dy);
  p.dh = static_cast<const moe::u32x4*>(dh);
  p.dx = static_cast<moe::u32x4*>(dx);
  p.dz = static_cast<moe::u32x4*>(dz);
  p.rows = rows;
  p.weight = row_weight;
  p.gate = gate;
  p.w_post = w_post;
  p.w_next = w_next;
  p.d_weight = d_row_weight;
  p.d_gate = d_gate;
  p.partial = static_cast<float*>(ws);
  p.n_valid = n_valid;
  p.d_err = d_err;
  p.z_rows = z_rows;
  p.T = static_cast<int>(T);
  p.H = static_cast<int>(H);
  p.groups = static_cast<int>(row / 16);
  p.k = k;
  p.scale = residual_scale;
  p.eps = eps;
  const moe::NormShape s = moe::norm_shape(moe::backward_blocks(T, p.groups), p.groups, moe::bwd_threads(k));
  if (T > 0) {
    moe::norm_launch<moe::Backward>(s, p, dtype, st);
    MOE_CHECK_LAUNCH();
  }
  const unsigned cols = static_cast<unsigned>((2 * H + moe::kWave - 1) / moe::kWave);
  moe::norm_weight_sum_kernel<<<cols, moe::kWave * moe::kSumRows, 0, st>>>(
      p.partial, T > 0 ? s.blocks : 0, p.H, dw_post, dw_next);
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}
