// Selective state space scan over a prompt, along one of the four scan directions.
//
// The recurrence of gtr_ssm.cuh is a chain over time for every (sequence, channel, state).
// Here a warp takes 64 / TL channels and TL x TS consecutive positions at once: each lane has TS
// consecutive positions of two neighbouring channels in registers, and for one state n after
// the other
//   1. computes its decays a_i = exp(delta_i A) and inputs b_i, and the state h that they give
//      from zero, with the product of the decays, P = exp(A sum delta_i);
//   2. joins (P, h) with the lanes before it by a shuffle scan over the TL lanes, the state
//      carried from the previous tile entering at the first lane;
//   3. runs its TS positions again from the state it now knows, with the same decays, and
//      adds C_i h_i to its outputs.
// Each exponential is computed once, and no chain is longer than TS plus log2(TL) steps, so
// the parallelism does not depend on the number of channels alone, and no block waits for
// another one.  A carried state meets TL - 1 lane products P and TS decays in a tile of TL TS
// positions: 15 to 39 approximate exponentials for 64 to 256 positions.  Each is off by up to
// 1e-7, and a constant step repeats its error, so it adds up linearly over a long memory: a
// state that lived through 16,384 positions of constant steps was off by up to 2.4e-4 of itself
// (4096 tokens of the step, one exponential each: 4.1e-4).
//
// Bound.  HBM asks for 8 bytes (16-bit data) per token and channel, 0.35 clocks an SM at the
// measured bandwidth; N = 16 exponentials at 16 a clock and SM are 1 clock, with P, softplus
// and SiLU 1.4; about 190 instructions at 128 a clock are 1.5, and shared memory and shuffles
// move about 1.3.  With three resources that near one another the kernels reach about half of
// each.  Measured (bf16, N = 16): eight 48 x 80 grids of 1536 channels 455 us (2.5 clocks a
// token and channel on each SM; one thread per state quadruple walking the sequence took 5.07
// ms), one 128 x 128 grid of 768 channels 273 us (20.3 ms), one 40 x 40 grid of 768 channels 31
// us (1.15 ms), two 64 x 64 grids of 1536 channels 170 us.  Measured and not kept: one channel
// a lane (555 us on the first of these: B and C are then read from shared memory twice as
// often), states in lanes and time in steps with two passes over time segments (700 us on the
// first, 245 us on the second).
#include <float.h>

#include <atomic>

#include "gtr_launch.cuh"
#include "gtr_ssm.cuh"
#include "gtr_ssm_host.h"
#include "gtr_sm100.cuh"
#include "gtr_vec.cuh"

namespace gtr {
namespace {

constexpr int kMaxSmem = 227 * 1024;  // of a block; an SM has 1 KB more and keeps 1 KB of each block
constexpr int kSms = 148;

// Copy `BYTES` (8 or 16) to shared memory asynchronously, or fill with zeros.
template <int BYTES>
__device__ __forceinline__ void copy_async(void* dst, const void* src, bool valid) {
  const uint32_t d = sm100::smem_u32(dst);
  const int n = valid ? BYTES : 0;
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(d), "l"(src), "r"(n) : "memory");
}

// Two neighbouring channels of a row.
template <typename T> struct Pair;
template <> struct Pair<__half> {
  static __device__ __forceinline__ float2 load(const void* p) { return __half22float2(*static_cast<const __half2*>(p)); }
  static __device__ __forceinline__ void store(void* p, float2 f) { *static_cast<__half2*>(p) = __floats2half2_rn(f.x, f.y); }
  using Raw = uint32_t;
};
template <> struct Pair<__nv_bfloat16> {
  static __device__ __forceinline__ float2 load(const void* p) {
    const uint32_t w = *static_cast<const uint32_t*>(p);
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  static __device__ __forceinline__ void store(void* p, float2 f) {
    *static_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(f.x, f.y);
  }
  using Raw = uint32_t;
};
template <> struct Pair<float> {
  static __device__ __forceinline__ float2 load(const void* p) { return *static_cast<const float2*>(p); }
  static __device__ __forceinline__ void store(void* p, float2 f) { *static_cast<float2*>(p) = f; }
  using Raw = uint2;
};

// The tile of TL x TS positions of CH channels in shared memory.  Raw rows are kept in TL
// blocks of TS rows with a gap between blocks: the lanes of a warp read the same row of every
// block at once, and the shift puts them on different banks.  Position t = l TS + 4 q + r of
// a table over positions is at place (q TL + l) 4 + r, the order of the lanes' 16-byte reads.
template <typename T, int TL, int TS, int CH>
struct Tile {
  static constexpr int kES = (int)sizeof(T);
  static constexpr int kTT = TL * TS;
  static constexpr int kRow = CH * kES;                            // bytes of a row of u, dt, z
  static constexpr int kBlock = TS * kRow + (kRow < 16 ? 8 : 16);  // one block of rows
  static constexpr int kRaw = (TL * kBlock + 15) / 16 * 16;        // u, dt or z
  static constexpr int kPiece = kRow < 16 ? kRow : 16;             // 8 bytes where a row has no more
  static constexpr int kPieces = kRow / kPiece;
  static constexpr int kN = 16 / kES;
  static constexpr int kPlaces = kTT + 4;  // of one state in a table

  static __host__ __device__ int n_block(int N) { return TS * N * kES + 16; }
  static __host__ __device__ int raw_n(int N) { return TL * n_block(N); }                 // B or C
  static __host__ __device__ int stage(int N) { return 3 * kRaw + 2 * raw_n(N); }
  static __host__ __device__ int spread(int N) { return 2 * N * kPlaces * 4; }            // B and C as fp32
  static __device__ __forceinline__ int position(int place) {
    return ((place / 4) % TL) * TS + (place / (4 * TL)) * 4 + place % 4;
  }
  static __device__ __forceinline__ int raw_at(int t) { return (t / TS) * kBlock + (t % TS) * kRow; }

  static __device__ __forceinline__ void set_tokens(const SsmParams& p, int* tok, int tile, int len, int tid, int threads) {
    for (int r = tid; r < kTT; r += threads) {
      const int s = tile * kTT + r;
      tok[r] = s < len ? p.map.token((unsigned)s) : -1;
    }
  }
  // Request a tile's rows; rows behind the sequence's end arrive as zeros.
  static __device__ __forceinline__ void load(const SsmParams& p, uint8_t* st, const int* tok, long long row0, int d0,
                                              int g, int tid, int threads) {
    for (int i = tid; i < kTT * kPieces; i += threads) {
      const int r = i / kPieces, q = i - r * kPieces;
      const int m = tok[r];
      const long long row = row0 + max(m, 0);
      uint8_t* dst = st + raw_at(r) + q * kPiece;
      const int e = d0 + q * (kPiece / kES);
      copy_async<kPiece>(dst, static_cast<const T*>(p.u) + row * p.u_ld + e, m >= 0);
      copy_async<kPiece>(dst + kRaw, static_cast<const T*>(p.dt) + row * p.dt_ld + e, m >= 0);
      if (p.z) copy_async<kPiece>(dst + 2 * kRaw, static_cast<const T*>(p.z) + row * p.z_ld + e, m >= 0);
    }
    const int np = p.N / kN, rn = raw_n(p.N);
    for (int r = tid; r < kTT; r += threads) {
      const int m = tok[r];
      const long long row = row0 + max(m, 0);
      uint8_t* dst = st + 3 * kRaw + (r / TS) * n_block(p.N) + (r % TS) * p.N * kES;
      const T* bm = static_cast<const T*>(p.Bm) + row * p.bm_ld + g * p.N;
      const T* cm = static_cast<const T*>(p.Cm) + row * p.cm_ld + g * p.N;
      for (int q = 0; q < np; ++q) {
        copy_async<16>(dst + 16 * q, bm + q * kN, m >= 0);
        copy_async<16>(dst + rn + 16 * q, cm + q * kN, m >= 0);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  // B and C as fp32, state by state.
  static __device__ __forceinline__ void spread_bc(int N, const uint8_t* st, float* table, int tid, int threads) {
    const int np = N / kN, rn = raw_n(N), nb = n_block(N);
    for (int i = tid; i < kTT * np; i += threads) {
      const int piece = i / kTT, k = i - piece * kTT;
      const int r = position(k);
      const uint8_t* src = st + 3 * kRaw + (r / TS) * nb + (r % TS) * N * kES + piece * 16;
      float f[kN], h[kN];
      Vec8<T>::load(*reinterpret_cast<const uint4*>(src), f);
      Vec8<T>::load(*reinterpret_cast<const uint4*>(src + rn), h);
      float* dst = table + piece * kN * kPlaces + k;
#pragma unroll
      for (int e = 0; e < kN; ++e) {
        dst[e * kPlaces] = f[e];
        dst[(N + e) * kPlaces] = h[e];
      }
    }
  }
};

// What a lane has of a tile: TS positions of two channels.
template <int TL, int TS>
struct Chains {
  float dl[2][TS], du[2][TS], y[2][TS], sum[2];

  // The decays of one state, and P.
  __device__ __forceinline__ void decays(const float* a_row, float2 (&a)[2][TS / 2], float (&P)[2]) const {
    const float2 A = *reinterpret_cast<const float2*>(a_row);
    P[0] = exp2_approx(sum[0] * A.x);
    P[1] = exp2_approx(sum[1] * A.y);
#pragma unroll
    for (int i = 0; i < TS / 2; ++i)
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const float2 e = mul2(make_float2(dl[v][2 * i], dl[v][2 * i + 1]), v ? make_float2(A.y, A.y) : make_float2(A.x, A.x));
        a[v][i] = make_float2(exp2_approx(e.x), exp2_approx(e.y));
      }
  }

  // One state: b_row, c_row this lane's B and C, h_row the carried state of its two channels,
  // next_row the following state's decay rates (NEXT): its exponentials are computed while
  // this state's shuffles and chains wait for one another.
  template <bool NEXT>
  __device__ __forceinline__ void state(int tl, const float4* b_row, const float4* c_row, float* h_row, const float* next_row,
                                        const float2 (&a)[2][TS / 2], float (&P)[2], float2 (&a_next)[2][TS / 2],
                                        float (&P_next)[2]) {
    float2 bb[2][TS / 2];
    const float2 old = *reinterpret_cast<const float2*>(h_row);
    const float in[2] = {old.x, old.y};
#pragma unroll
    for (int q = 0; q < TS / 4; ++q) {
      const float4 f = b_row[q * TL];
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        bb[v][2 * q] = mul2(make_float2(du[v][4 * q], du[v][4 * q + 1]), make_float2(f.x, f.y));
        bb[v][2 * q + 1] = mul2(make_float2(du[v][4 * q + 2], du[v][4 * q + 3]), make_float2(f.z, f.w));
      }
    }
    float h[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < TS / 2; ++i) {
#pragma unroll
      for (int v = 0; v < 2; ++v) h[v] = fmaf(a[v][i].x, h[v], bb[v][i].x);
#pragma unroll
      for (int v = 0; v < 2; ++v) h[v] = fmaf(a[v][i].y, h[v], bb[v][i].y);
    }
    if (tl == 0) {
      h[0] = fmaf(P[0], in[0], h[0]);
      h[1] = fmaf(P[1], in[1], h[1]);
    }
    __syncwarp();  // every lane has the old carry
    if constexpr (NEXT) decays(next_row, a_next, P_next);
#pragma unroll
    for (int s = 1; s < TL; s *= 2) {
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const float hp = __shfl_up_sync(0xffffffffu, h[v], s * (32 / TL));
        if (tl >= s) h[v] = fmaf(P[v], hp, h[v]);
        if (2 * s < TL) {
          const float Pp = __shfl_up_sync(0xffffffffu, P[v], s * (32 / TL));
          if (tl >= s) P[v] *= Pp;
        }
      }
    }
    float x[2];
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      const float hp = __shfl_up_sync(0xffffffffu, h[v], 32 / TL);
      x[v] = tl > 0 ? hp : in[v];
    }
#pragma unroll
    for (int q = 0; q < TS / 4; ++q) {
      const float4 f = c_row[q * TL];
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        float2 h0, h1;
        h0.x = fmaf(a[v][2 * q].x, x[v], bb[v][2 * q].x);
        h0.y = fmaf(a[v][2 * q].y, h0.x, bb[v][2 * q].y);
        h1.x = fmaf(a[v][2 * q + 1].x, h0.y, bb[v][2 * q + 1].x);
        h1.y = x[v] = fmaf(a[v][2 * q + 1].y, h1.x, bb[v][2 * q + 1].y);
        const float2 y0 = fma2(h0, make_float2(f.x, f.y), make_float2(y[v][4 * q], y[v][4 * q + 1]));
        const float2 y1 = fma2(h1, make_float2(f.z, f.w), make_float2(y[v][4 * q + 2], y[v][4 * q + 3]));
        y[v][4 * q] = y0.x, y[v][4 * q + 1] = y0.y, y[v][4 * q + 2] = y1.x, y[v][4 * q + 3] = y1.y;
      }
    }
    if (tl == TL - 1) *reinterpret_cast<float2*>(h_row) = make_float2(x[0], x[1]);
  }

  // The states n0, n0 + step, ... of N: tables of the tile, rows of CH channels, this lane's
  // first channel c.
  template <int CH>
  __device__ __forceinline__ void states(int N, int n0, int step, int tl, int c, const float* table, const float* a_table,
                                         float* carry) {
    constexpr int kPlaces = TL * TS + 4;
    float2 a0[2][TS / 2], a1[2][TS / 2];
    float P0[2], P1[2];
    const auto b_row = [&](int n) { return reinterpret_cast<const float4*>(table + n * kPlaces) + tl; };
    const auto c_row = [&](int n) { return reinterpret_cast<const float4*>(table + (N + n) * kPlaces) + tl; };
    decays(a_table + n0 * CH + c, a0, P0);
    for (int n = n0;; n += 2 * step) {
      const int m = n + step;
      if (m >= N) {
        state<false>(tl, b_row(n), c_row(n), carry + n * CH + c, nullptr, a0, P0, a1, P1);
        break;
      }
      state<true>(tl, b_row(n), c_row(n), carry + n * CH + c, a_table + m * CH + c, a0, P0, a1, P1);
      if (m + step >= N) {
        state<false>(tl, b_row(m), c_row(m), carry + m * CH + c, nullptr, a1, P1, a0, P0);
        break;
      }
      state<true>(tl, b_row(m), c_row(m), carry + m * CH + c, a_table + (m + step) * CH + c, a1, P1, a0, P0);
    }
  }
};

// A log2(e), held finite.  A rate of -inf, or one that the factor takes out of fp32's range, forgets
// at once either way, but the positions behind a sequence's end in its last tile have steps of 0
// and must keep the state: exp2(0 * -inf) would be a NaN.  A NaN stays one.
__device__ __forceinline__ float log2_rate(float a) {
  const float r = a * kLog2e;
  return fabsf(r) > FLT_MAX ? copysignf(FLT_MAX, r) : r;
}

// The tables that live as long as the block, [N][CH]: A log2(e) and the carried states.
template <int CH>
__device__ __forceinline__ void load_tables(const SsmParams& p, float* a_table, float* carry, int d0, int b, int tid,
                                            int threads) {
  for (int i = tid; i < p.N * CH; i += threads) {
    const int ch = i / p.N, n = i - ch * p.N;
    a_table[n * CH + ch] = log2_rate(__ldg(p.A + (long long)(d0 + ch) * p.N + n));
    carry[n * CH + ch] = p.state_in ? p.state_in[((long long)b * p.D + d0 + ch) * p.N + n] : 0.f;
  }
}
template <int CH>
__device__ __forceinline__ void store_states(const SsmParams& p, const float* carry, int d0, int b, int tid, int threads) {
  for (int i = tid; i < p.N * CH; i += threads) {
    const int ch = i / p.N, n = i - ch * p.N;
    p.state_out[((long long)b * p.D + d0 + ch) * p.N + n] = carry[n * CH + ch];
  }
}
__device__ __forceinline__ float2 channel_pair(const float* v, int ch) {
  return v ? make_float2(__ldg(v + ch), __ldg(v + ch + 1)) : make_float2(0.f, 0.f);
}
__device__ __forceinline__ int sequence_length(const SsmParams& p, int b) {
  return p.lengths ? min(max(__ldg(p.lengths + b), 0), p.L) : p.L;
}

// ------------------------------------------------------------------------------- many channels
// WC warps of 64 / TL channels each: every warp does all states of its channels, and the phases
// of one block (copies, tables, states, outputs) overlap with those of the other blocks on
// the SM.
template <typename T, int TL, int TS, int WC>
struct WideLayout {
  using Tl = Tile<T, TL, TS, WC * 64 / TL>;
  int spread, hold, tokens, table, total;  // the raw tile is at 0
  __host__ __device__ explicit WideLayout(int N) {
    spread = Tl::stage(N);
    hold = spread + Tl::spread(N);  // z, then the outputs
    tokens = hold + Tl::kRaw;       // [3][kTT]: next, this, last tile
    table = tokens + 3 * Tl::kTT * 4;
    total = table + 2 * N * (WC * 64 / TL) * 4;
  }
};

template <typename T, int TL, int TS, int WC, int MB>
__global__ void __launch_bounds__(32 * WC, MB) ssm_scan_wide_kernel(const SsmParams p) {
  constexpr int kThreads = 32 * WC, kCh = WC * 64 / TL;
  using Tl = Tile<T, TL, TS, kCh>;
  constexpr int kTT = Tl::kTT, kES = Tl::kES, kPiece = Tl::kPiece, kPieces = Tl::kPieces;
  extern __shared__ __align__(128) uint8_t smem[];
  const WideLayout<T, TL, TS, WC> lay(p.N);
  float* table = reinterpret_cast<float*>(smem + lay.spread);
  int* tokens = reinterpret_cast<int*>(smem + lay.tokens);
  float* a_table = reinterpret_cast<float*>(smem + lay.table);
  float* carry = a_table + p.N * kCh;
  const int tid = threadIdx.x, lane = tid & 31;
  // lanes of one time lane are neighbours: their 16-byte reads of B and C are the same, and the
  // shared memory answers them in half the time that it takes for repeats eight lanes apart
  const int tl = lane / (32 / TL);
  const int c = ((tid >> 5) * (32 / TL) + lane % (32 / TL)) * 2;  // the first of this lane's channels
  const int d0 = blockIdx.x * kCh, b = blockIdx.y;
  const int g = d0 / (p.D / p.G);
  const long long row0 = (long long)b * p.L;

  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int len = sequence_length(p, b), tiles = (len + kTT - 1) / kTT;
  load_tables<kCh>(p, a_table, carry, d0, b, tid, kThreads);
  if (tiles > 0) {
    Tl::set_tokens(p, tokens, 0, len, tid, kThreads);
    __syncthreads();
    Tl::load(p, smem, tokens, row0, d0, g, tid, kThreads);
  }
  const float2 skip = channel_pair(p.skip, d0 + c), bias = channel_pair(p.dt_bias, d0 + c);
  const uint8_t* raw = smem + tl * Tl::kBlock + c * kES;
  uint8_t* hold = smem + lay.hold + tl * Tl::kBlock + c * kES;
  for (int tile = 0; tile < tiles; ++tile) {
    const bool more = tile + 1 < tiles;
    const int* tok = tokens + (tile % 3) * kTT;
    int* tok_next = tokens + ((tile + 1) % 3) * kTT;
    if (more) Tl::set_tokens(p, tok_next, tile + 1, len, tid, kThreads);
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();  // the tile is here, its predecessor's outputs have left, tokens are set
    Tl::spread_bc(p.N, smem, table, tid, kThreads);
    Chains<TL, TS> ch;
#pragma unroll
    for (int i = 0; i < TS; ++i) {
      const float2 x = Pair<T>::load(raw + Tl::kRaw + i * Tl::kRow);
      ch.dl[0][i] = x.x + bias.x;
      ch.dl[1][i] = x.y + bias.y;
    }
    if (p.softplus) {  // one branch around them all, so that they overlap
#pragma unroll
      for (int i = 0; i < TS; ++i) {
        ch.dl[0][i] = softplus_f32(ch.dl[0][i]);
        ch.dl[1][i] = softplus_f32(ch.dl[1][i]);
      }
    }
    const int left = len - tile * kTT - tl * TS;  // positions of the sequence from here on
    ch.sum[0] = ch.sum[1] = 0.f;
#pragma unroll
    for (int i = 0; i < TS; ++i) {
      const float2 u = Pair<T>::load(raw + i * Tl::kRow);
      if (i >= left) ch.dl[0][i] = ch.dl[1][i] = 0.f;
      ch.du[0][i] = ch.dl[0][i] * u.x;
      ch.du[1][i] = ch.dl[1][i] * u.y;
      ch.y[0][i] = skip.x * u.x;
      ch.y[1][i] = skip.y * u.y;
      ch.sum[0] += ch.dl[0][i];
      ch.sum[1] += ch.dl[1][i];
    }
    if (p.z) {
      using Raw = typename Pair<T>::Raw;
#pragma unroll
      for (int i = 0; i < TS; ++i)
        *reinterpret_cast<Raw*>(hold + i * Tl::kRow) = *reinterpret_cast<const Raw*>(raw + 2 * Tl::kRaw + i * Tl::kRow);
    }
    __syncthreads();  // B and C are spread, the raw tile has been read
    if (more) Tl::load(p, smem, tok_next, row0, d0, g, tid, kThreads);
    ch.template states<kCh>(p.N, 0, 1, tl, c, table, a_table, carry);
    if (p.z) {
#pragma unroll
      for (int i = 0; i < TS; ++i) {
        const float2 z = Pair<T>::load(hold + i * Tl::kRow);
        ch.y[0][i] *= silu_f32(z.x);
        ch.y[1][i] *= silu_f32(z.y);
      }
    }
#pragma unroll
    for (int i = 0; i < TS; ++i) Pair<T>::store(hold + i * Tl::kRow, make_float2(ch.y[0][i], ch.y[1][i]));
    __syncthreads();  // the outputs are there; the spread B and C have been read
    for (int i = tid; i < kTT * kPieces; i += kThreads) {
      const int r = i / kPieces, q = i - r * kPieces;
      const int m = tok[r];
      if (m < 0) continue;
      const uint8_t* src = smem + lay.hold + Tl::raw_at(r) + q * kPiece;
      T* dst = static_cast<T*>(p.out) + (row0 + m) * p.D + d0 + q * (kPiece / kES);
      if constexpr (kPiece == 16)
        *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(src);
      else
        *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<const uint2*>(src);
    }
  }
  if (p.state_out) {
    __syncthreads();
    store_states<kCh>(p, carry, d0, b, tid, kThreads);
  }
}

// -------------------------------------------------------------------------------- few channels
// One block on an SM: WC groups of channels times SG groups of states, a warp each, run the
// states of one tile while WP other warps copy and prepare the next one (B, C, delta and delta
// u as fp32 tables) and finish the last one (the sum over the state groups, skip, gate).
// Tables and partial outputs are doubled, raw tiles (u and z are read again at the end) are three; the two sides meet at named barriers: ready[k & 1]
// (tile k's tables are there; partial outputs k - 2 have been read) and done[k & 1] (partial
// outputs k are there; tile k's tables have been read).
template <typename T, int TL, int TS, int WC, int SG>
struct DeepLayout {
  static constexpr int kCh = WC * 64 / TL;
  using Tl = Tile<T, TL, TS, kCh>;
  // of one channel: the channels that eight lanes read 16 bytes of at once are on other banks
  static constexpr int kStride = Tl::kTT + (TL == 16 ? 8 : 4);
  static constexpr int kDelta = 2 * kCh * kStride * 4;  // delta and delta u
  static constexpr int kPart = SG * kCh * kStride * 4;
  int stage, spread, delta, part, tokens, table, total;  // [3] raw stages at 0
  __host__ __device__ explicit DeepLayout(int N) {
    stage = Tl::stage(N);
    spread = 3 * stage;                      // [2]
    delta = spread + 2 * Tl::spread(N);      // [2]
    part = delta + 2 * kDelta;               // [2]
    tokens = part + 2 * kPart;               // [4][kTT]
    table = tokens + 4 * Tl::kTT * 4;
    total = table + 2 * N * kCh * 4;
  }
};

template <int THREADS>
__device__ __forceinline__ void bar_sync(int id) {
  asm volatile("barrier.sync %0, %1;" ::"r"(id), "n"(THREADS) : "memory");
}
template <int THREADS>
__device__ __forceinline__ void bar_arrive(int id) {
  asm volatile("barrier.arrive %0, %1;" ::"r"(id), "n"(THREADS) : "memory");
}

template <typename T, int TL, int TS, int WC, int SG, int WP>
__global__ void __launch_bounds__(32 * (WC * SG + WP), 1) ssm_scan_deep_kernel(const SsmParams p) {
  constexpr int kCh = WC * 64 / TL;
  constexpr int kPrep = 32 * WP, kAll = 32 * (WC * SG + WP);
  constexpr int kReady = 1, kDone = 3, kPrepBar = 5;  // barrier numbers; ready and done: + (tile & 1)
  using Tl = Tile<T, TL, TS, kCh>;
  using Lay = DeepLayout<T, TL, TS, WC, SG>;
  constexpr int kTT = Tl::kTT, kES = Tl::kES, kStride = Lay::kStride;
  extern __shared__ __align__(128) uint8_t smem[];
  const Lay lay(p.N);
  int* tokens = reinterpret_cast<int*>(smem + lay.tokens);
  float* a_table = reinterpret_cast<float*>(smem + lay.table);
  float* carry = a_table + p.N * kCh;
  const int tid = threadIdx.x;
  const int d0 = blockIdx.x * kCh, b = blockIdx.y;
  const int g = d0 / (p.D / p.G);
  const long long row0 = (long long)b * p.L;
  const int spread_bytes = Tl::spread(p.N);

  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int len = sequence_length(p, b), tiles = (len + kTT - 1) / kTT;
  load_tables<kCh>(p, a_table, carry, d0, b, tid, kAll);
  __syncthreads();

  if (tid < kPrep) {
    // the channels that this thread prepares and finishes, and their places in a tile
    constexpr int kRows = kPrep / (kCh / 2), kIter = kTT / kRows;
    static_assert(kTT % kRows == 0, "whole turns");
    const int pc = 2 * (tid % (kCh / 2)), k0 = tid / (kCh / 2);
    const float2 skip = channel_pair(p.skip, d0 + pc), bias = channel_pair(p.dt_bias, d0 + pc);
    if (tiles > 0) {
      Tl::set_tokens(p, tokens, 0, len, tid, kPrep);
      bar_sync<kPrep>(kPrepBar);
      Tl::load(p, smem, tokens, row0, d0, g, tid, kPrep);
    }
    for (int tile = 0; tile <= tiles; ++tile) {
      if (tile < tiles) {
        const uint8_t* st = smem + (tile % 3) * lay.stage;
        const bool more = tile + 1 < tiles;
        int* tok_next = tokens + ((tile + 1) & 3) * kTT;
        if (more) Tl::set_tokens(p, tok_next, tile + 1, len, tid, kPrep);
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        bar_sync<kPrep>(kPrepBar);  // the tile is here, tokens are set, tile - 2 is finished
        if (more) Tl::load(p, smem + ((tile + 1) % 3) * lay.stage, tok_next, row0, d0, g, tid, kPrep);
        Tl::spread_bc(p.N, st, reinterpret_cast<float*>(smem + lay.spread + (tile & 1) * spread_bytes), tid, kPrep);
        float* delta = reinterpret_cast<float*>(smem + lay.delta + (tile & 1) * Lay::kDelta);
        float2 x[kIter], u[kIter];
#pragma unroll
        for (int i = 0; i < kIter; ++i) {
          const uint8_t* at = st + Tl::raw_at(Tl::position(k0 + i * kRows)) + pc * kES;
          u[i] = Pair<T>::load(at);
          x[i] = add2(Pair<T>::load(at + Tl::kRaw), bias);
        }
        if (p.softplus) {  // one branch around them all, so that they overlap
#pragma unroll
          for (int i = 0; i < kIter; ++i) x[i] = make_float2(softplus_f32(x[i].x), softplus_f32(x[i].y));
        }
#pragma unroll
        for (int i = 0; i < kIter; ++i) {
          const int k = k0 + i * kRows;
          if (tile * kTT + Tl::position(k) >= len) x[i] = make_float2(0.f, 0.f);
          const float2 du = mul2(x[i], u[i]);
          delta[pc * kStride + k] = x[i].x;
          delta[(pc + 1) * kStride + k] = x[i].y;
          delta[(kCh + pc) * kStride + k] = du.x;
          delta[(kCh + pc + 1) * kStride + k] = du.y;
        }
        bar_arrive<kAll>(kReady + (tile & 1));
      }
      if (tile > 0) {  // finish the last tile
        const int last = tile - 1;
        const uint8_t* st = smem + (last % 3) * lay.stage;
        const int* tok = tokens + (last & 3) * kTT;
        const float* part = reinterpret_cast<const float*>(smem + lay.part + (last & 1) * Lay::kPart);
        bar_sync<kAll>(kDone + (last & 1));
        float2 v[kIter], z[kIter];
#pragma unroll
        for (int i = 0; i < kIter; ++i) {
          const int k = k0 + i * kRows;
          const uint8_t* at = st + Tl::raw_at(Tl::position(k)) + pc * kES;
          z[i] = Pair<T>::load(at + 2 * Tl::kRaw);
          v[i] = mul2(skip, Pair<T>::load(at));
#pragma unroll
          for (int s = 0; s < SG; ++s)
            v[i] = add2(v[i], make_float2(part[(s * kCh + pc) * kStride + k], part[(s * kCh + pc + 1) * kStride + k]));
        }
        if (p.z) {
#pragma unroll
          for (int i = 0; i < kIter; ++i) v[i] = mul2(v[i], silu2(z[i]));
        }
#pragma unroll
        for (int i = 0; i < kIter; ++i) {
          const int m = tok[Tl::position(k0 + i * kRows)];
          if (m >= 0) Pair<T>::store(static_cast<T*>(p.out) + (row0 + m) * p.D + d0 + pc, v[i]);
        }
      }
    }
  } else {
    const int lane = tid & 31, warp = (tid - kPrep) >> 5;
    const int tl = lane / (32 / TL);
    const int c = ((warp % WC) * (32 / TL) + lane % (32 / TL)) * 2;
    const int sg = warp / WC;
    for (int tile = 0; tile < tiles; ++tile) {
      bar_sync<kAll>(kReady + (tile & 1));
      const float* delta = reinterpret_cast<const float*>(smem + lay.delta + (tile & 1) * Lay::kDelta);
      Chains<TL, TS> ch;
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        ch.sum[v] = 0.f;
#pragma unroll
        for (int q = 0; q < TS / 4; ++q) {
          const float4 f = *reinterpret_cast<const float4*>(delta + (c + v) * kStride + (q * TL + tl) * 4);
          const float4 h = *reinterpret_cast<const float4*>(delta + (kCh + c + v) * kStride + (q * TL + tl) * 4);
          ch.dl[v][4 * q] = f.x, ch.dl[v][4 * q + 1] = f.y, ch.dl[v][4 * q + 2] = f.z, ch.dl[v][4 * q + 3] = f.w;
          ch.du[v][4 * q] = h.x, ch.du[v][4 * q + 1] = h.y, ch.du[v][4 * q + 2] = h.z, ch.du[v][4 * q + 3] = h.w;
          ch.sum[v] += (f.x + f.y) + (f.z + f.w);
          ch.y[v][4 * q] = ch.y[v][4 * q + 1] = ch.y[v][4 * q + 2] = ch.y[v][4 * q + 3] = 0.f;
        }
      }
      ch.template states<kCh>(p.N, sg, SG, tl, c, reinterpret_cast<const float*>(smem + lay.spread + (tile & 1) * spread_bytes),
                              a_table, carry);
      float* part = reinterpret_cast<float*>(smem + lay.part + (tile & 1) * Lay::kPart) + sg * kCh * kStride;
#pragma unroll
      for (int v = 0; v < 2; ++v)
#pragma unroll
        for (int q = 0; q < TS / 4; ++q)
          *reinterpret_cast<float4*>(part + (c + v) * kStride + (q * TL + tl) * 4) =
              make_float4(ch.y[v][4 * q], ch.y[v][4 * q + 1], ch.y[v][4 * q + 2], ch.y[v][4 * q + 3]);
      bar_arrive<kAll>(kDone + (tile & 1));
    }
  }
  if (p.state_out) {
    __syncthreads();
    store_states<kCh>(p, carry, d0, b, tid, kAll);
  }
}

// The kernel may use kMaxSmem on the current device: asked for once per device and kernel
// (`done`, a bit for each device).
template <typename K>
bool allow_smem(K* kernel, std::atomic<unsigned long long>& done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return true;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem) != cudaSuccess) return false;
  done.fetch_or(bit, std::memory_order_relaxed);
  return true;
}

template <typename T, int TL, int TS, int WC, int MB>
gtr_status_t launch_wide(const SsmParams& p, cudaStream_t stream) {
  static std::atomic<unsigned long long> allowed{0};
  if (!allow_smem(ssm_scan_wide_kernel<T, TL, TS, WC, MB>, allowed)) return cuda_failed();
  constexpr int kCh = WC * 64 / TL;
  // Blocks that leave room on the SMs are spread evenly by asking for as much shared memory as
  // lets no SM take more than its share: next to blocks of a kernel that still runs they would
  // be packed on part of the SMs (144 blocks of <32, 8> then took the time of 432, 84 us, and 50
  // us when spread)
  const int need = WideLayout<T, TL, TS, WC>(p.N).total;
  const long long share = ((long long)p.B * (p.D / kCh) + kSms - 1) / kSms;
  const int even = share <= MB ? (kMaxSmem + 1024) / (int)share - 1024 : 0;
  return launch_serial(ssm_scan_wide_kernel<T, TL, TS, WC, MB>, dim3((unsigned)(p.D / kCh), (unsigned)p.B), dim3(32 * WC),
                       (size_t)(need > even ? need : even), stream, p);
}
template <typename T, int TL, int TS, int WC, int SG, int WP>
gtr_status_t launch_deep(const SsmParams& p, cudaStream_t stream) {
  static std::atomic<unsigned long long> allowed{0};
  if (!allow_smem(ssm_scan_deep_kernel<T, TL, TS, WC, SG, WP>, allowed)) return cuda_failed();
  constexpr int kCh = WC * 64 / TL;
  return launch_serial(ssm_scan_deep_kernel<T, TL, TS, WC, SG, WP>, dim3((unsigned)(p.D / kCh), (unsigned)p.B),
                       dim3(32 * (WC * SG + WP)), (size_t)DeepLayout<T, TL, TS, WC, SG>(p.N).total, stream, p);
}

// The plan.  Each kernel holds a number of blocks on an SM, and one that has some left over for
// another wave pays for it whole, so the plans are compared by what their waves take: `one` and
// `most` are the measured microseconds of 2048 positions (bf16, N = 16) with one block on each
// SM and with as many as it holds; in between they are taken as evenly spaced, and everything
// scales with the positions, whole tiles of them, and with N but for a share (two sequences of
// 4096 positions and 768 channels, N = 64: deep<8> over 64 positions 420 us, wide<16, 8> 499 us).
// Measured with the plan taken and the next best (2048 positions each, B D / 8 = W):
//   W = 144  deep 36, wide<32, 8> 50;            W = 288  wide<32, 8> 67, wide<16, 16> 69, deep 72
//   W = 432  wide<32, 8> 86, wide<16, 16> 91;    W = 576  wide<16, 16> 92, wide<16, 8> 106
//   W = 880  wide<16, 8> 139, wide<16, 16> 154;  W = 1152 wide<8, 16> 164, wide<16, 16> 182
//   W = 1728 wide<8, 8> 247, wide<8, 16> 268
// Other types and N take the same figures; against every other plan on 16 shapes of fp32 and of N =
// 8, 32 and 64 the choice was the quickest but for two fp32 ones (two sequences of 4096 positions
// and 1536 channels: deep<8> 237 us, wide<16, 8> 224 us; four of 2048 and 864: 124 and 114 us).
// The lengths of a padded batch are on the device; its blocks are counted half, as if the
// lengths were spread evenly (three sequences of 416 channels, one full, one of some tokens, one
// empty: deep 27 us, a plan for all of them at once 56 us).  A batch that comes with lengths and
// is full pays for that: with and without them eight sequences of 1600 positions and 768 channels
// 147 and 112 us, four of 4096 and 1536 335 and 272 us, four of 1600 and 768 89 and 76 us, eight of
// 3840 and 1536 498 and 453 us.
struct ScanPlan {
  int channels, positions;  // of a block's tile
  int holds;                // blocks on an SM where shared memory allows it
  float one, most;
  float fixed;              // share of that which does not grow with N
};
enum { kDeep4, kDeep8, kDeep8Short, kWide32x8, kWide16x16, kWide16x8, kWide8x16, kWide8x8, kPlans };
static_assert(GTR_SSM_DEEP_4 == kDeep4 + 1 && GTR_SSM_WIDE_8X8 == kWide8x8 + 1, "the header's plans, in this order");
constexpr ScanPlan kScanPlans[kPlans] = {
    {4, 128, 1, 28.f, 28.f, .36f},   {8, 128, 1, 36.f, 36.f, .36f},  {8, 64, 1, 41.f, 41.f, .48f},
    {8, 256, 3, 50.f, 86.f, .29f},   {16, 256, 2, 69.f, 91.f, .29f}, {16, 128, 3, 80.f, 139.f, .29f},
    {32, 128, 2, 116.f, 163.f, .29f}, {32, 64, 3, 139.f, 247.f, .29f},
};

float plan_cost(const SsmParams& p, int plan, int smem) {
  constexpr float kNever = 3e38f;
  const ScanPlan& s = kScanPlans[plan];
  const int fits = (kMaxSmem + 1024) / (smem + 1024);
  if (smem > kMaxSmem || p.D / p.G % s.channels != 0) return kNever;
  const int holds = fits < s.holds ? fits : s.holds;
  const auto wave = [&](long long blocks) {  // microseconds with so many blocks on an SM
    return blocks == 0 ? 0.f : s.one + (s.holds > 1 ? (s.most - s.one) * (float)(blocks - 1) / (float)(s.holds - 1) : 0.f);
  };
  const long long all = (long long)p.B * (p.D / s.channels), blocks = p.lengths ? (all + 1) / 2 : all;
  const long long slots = (long long)kSms * holds;
  const long long tiles = ((long long)p.L + s.positions - 1) / s.positions;
  return ((float)(blocks / slots) * wave(holds) + wave((blocks % slots + kSms - 1) / kSms)) *
         (s.fixed + (1.f - s.fixed) * (float)p.N / 16.f) * (float)(tiles * s.positions);
}

// Prompts that leave a tile mostly empty walk token by token instead (gtr_ssm_step.cu).  Measured
// (1536 channels), walk and the quickest tiles: bf16, N = 16, 512 sequences of 24 tokens 377 and 514
// us, of 32 496 and 516 us; 16 sequences of 24 17 and 21 us, of 32 26 and 21 us; 4 sequences of 8
// 5.2 and 8.3 us, of 12 7.2 and 8.4 us, of 16 9.3 and 8.4 us.  fp32: 512 of 24 341 and 543 us, 16 of
// 24 20 and 23 us, 4 of 8 3.9 and 8.8 us.  The tiles grow faster with N than the walk: N = 64, bf16,
// 512 of 24 698 and 2153 us, of 32 918 and 2163 us; 16 of 32 45 and 81 us; 4 of 12 9.0 and 27 us,
// past the border of this rule, which looks at lengths and channels alone.
bool few_tokens(const SsmParams& p) {
  const long long channels = (long long)p.B * p.D;
  return channels >= 16384 ? p.L <= 24 : channels >= 4096 && p.L <= 8;
}

template <typename T>
int choose_plan(const SsmParams& p) {
  const int smem[kPlans] = {DeepLayout<T, 16, 8, 1, 8>(p.N).total, DeepLayout<T, 16, 8, 2, 4>(p.N).total,
                            DeepLayout<T, 8, 8, 1, 8>(p.N).total,  WideLayout<T, 32, 8, 4>(p.N).total,
                            WideLayout<T, 16, 16, 4>(p.N).total,   WideLayout<T, 16, 8, 4>(p.N).total,
                            WideLayout<T, 8, 16, 4>(p.N).total,    WideLayout<T, 8, 8, 4>(p.N).total};
  int best = kWide16x8;  // fits for every N and type
  float least = plan_cost(p, best, smem[best]);
  for (int i = 0; i < kPlans; ++i) {
    const float c = plan_cost(p, i, smem[i]);
    if (c < least) best = i, least = c;
  }
  return best;
}

template <typename T>
gtr_status_t launch_scan_t(const SsmParams& p, cudaStream_t stream) {
  switch (choose_plan<T>(p)) {
    case kDeep4: return launch_deep<T, 16, 8, 1, 8, 8>(p, stream);
    case kDeep8: return launch_deep<T, 16, 8, 2, 4, 8>(p, stream);
    case kDeep8Short: return launch_deep<T, 8, 8, 1, 8, 8>(p, stream);
    case kWide32x8: return launch_wide<T, 32, 8, 4, 3>(p, stream);
    case kWide16x16: return launch_wide<T, 16, 16, 4, 2>(p, stream);
    case kWide8x16: return launch_wide<T, 8, 16, 4, 2>(p, stream);
    case kWide8x8: return launch_wide<T, 8, 8, 4, 3>(p, stream);
    default: return launch_wide<T, 16, 8, 4, 3>(p, stream);
  }
}

}  // namespace
}  // namespace gtr

extern "C" gtr_status_t gtr_ssm_scan(const void* u, int64_t u_ld, const void* dt, int64_t dt_ld, const float* A,
                                     const void* Bm, int64_t bm_ld, const void* Cm, int64_t cm_ld, const void* z,
                                     int64_t z_ld, const float* skip, const float* dt_bias, int softplus,
                                     const float* state_in, float* state_out, const int* lengths, void* out, int B,
                                     int grid_H, int grid_W, int D, int N, int G, int direction, int dtype,
                                     gtr_stream_t stream) {
  using namespace gtr;
  SsmParams p{u,    dt,      Bm,       Cm,        z,       u_ld, dt_ld, bm_ld, cm_ld, z_ld, A,
              skip, dt_bias, state_in, state_out, lengths, out,  B,     0,     D,     N,    G,
              softplus != 0, ScanMap{1, 1, 0, 1}};
  const gtr_status_t st = validate_ssm(p, grid_H, grid_W, direction, dtype);
  if (st != GTR_OK) return st;
  p.L = grid_H * grid_W;
  p.map = ScanMap::make(direction, grid_H, grid_W);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (few_tokens(p)) return launch_ssm_walk(p, dtype, s);
  switch (dtype) {
    case GTR_F16: return launch_scan_t<__half>(p, s);
    case GTR_BF16: return launch_scan_t<__nv_bfloat16>(p, s);
    default: return launch_scan_t<float>(p, s);
  }
}

extern "C" gtr_status_t gtr_ssm_scan_plan(int B, int grid_H, int grid_W, int D, int N, int G, int dtype, int padded,
                                          int* plan) {
  using namespace gtr;
  const gtr_status_t st = validate_ssm_shape(B, grid_H, grid_W, D, N, G, dtype);
  if (st != GTR_OK) return st;
  if (!plan) return GTR_ERR_INVALID_ARG;
  SsmParams p{};
  p.B = B, p.L = grid_H * grid_W, p.D = D, p.N = N, p.G = G;
  p.lengths = padded ? &p.B : nullptr;  // only whether there are any counts
  if (few_tokens(p)) {
    *plan = GTR_SSM_WALK;
    return GTR_OK;
  }
  switch (dtype) {
    case GTR_F16: *plan = 1 + choose_plan<__half>(p); break;
    case GTR_BF16: *plan = 1 + choose_plan<__nv_bfloat16>(p); break;
    default: *plan = 1 + choose_plan<float>(p);
  }
  return GTR_OK;
}
