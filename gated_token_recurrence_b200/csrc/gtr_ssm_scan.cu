// Selective state space scan over a prompt, along one of the four scan directions.
//
// The recurrence of gtr_ssm.cuh is a chain over time for every (sequence, channel, state).
// Here a warp takes CW = 32 / TL channels and TL x TS consecutive positions at once: each lane
// has TS consecutive positions of one channel in registers, and for one state n after the
// other
//   1. computes its TS decays a_i = exp(delta_i A) and inputs b_i, and the state h that they
//      give from zero, with the product of the decays, P = exp(A sum delta_i);
//   2. joins (P, h) with the lanes before it by a shuffle scan over the TL lanes, the state
//      carried from the previous tile entering at the first lane;
//   3. runs its TS positions again from the state it now knows, with the same decays, and
//      adds C_i h_i to its outputs.
// Each exponential is computed once, and no chain is longer than TS plus log2(TL) steps, so
// the parallelism does not depend on the number of channels alone, and no block waits for
// another one.  The decays inside a lane enter products of at most TS factors; across lanes
// and tiles one P stands for TS of them, so the approximate exponential's bias (2e-8) does
// not build up over a long memory.
//
// A CTA of four warps covers 4 CW channels of one sequence and walks along it in tiles of
// TL x TS positions: rows come in by cp.async (the direction only changes which row comes
// next; rows behind the sequence's end arrive as zeros), B and C are spread once per tile as
// fp32 in the order in which the lanes read them, outputs return through the place of u.
//
// Bound: the exponential unit.  N exponentials per token and channel at 16 a clock and SM are
// N / 16 clocks, against 0.35 clocks for the 8 bytes of u, dt, z and out (16-bit data) at the
// measured HBM bandwidth.
#include <mutex>

#include "gtr_launch.cuh"
#include "gtr_ssm.cuh"
#include "gtr_ssm_host.h"
#include "gtr_sm100.cuh"
#include "gtr_vec.cuh"

namespace gtr {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;

// Shared memory of one CTA.  Rows of a tile are kept in TL blocks of TS rows with 16 bytes
// between blocks: the lanes of a warp read the same row of every block at once, and the shift
// puts them on different banks.
template <int ES, int TL, int TS>
struct Layout {
  int ch_block, n_block;      // bytes from one block of rows to the next: u, dt, z; B, C
  int ch_tile, n_tile;        // bytes of one tensor's tile
  int stage;                  // bytes of one stage: u, dt, z, B, C
  int spread, tokens, table;  // offsets of the fp32 B and C, the token indices, A and carry
  int total;
  __host__ __device__ Layout(int N, int stages) {
    constexpr int kCh = kWarps * 32 / TL;
    ch_block = TS * kCh * ES + 16;
    n_block = TS * N * ES + 16;
    ch_tile = TL * ch_block;
    n_tile = TL * n_block;
    stage = 3 * ch_tile + 2 * n_tile;
    spread = stages * stage;
    tokens = spread + 2 * N * (TL * TS + 4) * 4;
    table = tokens + 3 * TL * TS * 4;
    total = table + 2 * N * kCh * 4;
  }
};

// Copy `bytes` (8 or 16) to shared memory asynchronously, or fill with zeros.
template <int BYTES>
__device__ __forceinline__ void copy_async(void* dst, const void* src, bool valid) {
  const uint32_t d = sm100::smem_u32(dst);
  const int n = valid ? BYTES : 0;
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(d), "l"(src), "r"(n) : "memory");
}

template <typename T, int TL, int TS, int NU>
__global__ void __launch_bounds__(kThreads) ssm_scan_kernel(const SsmParams p, const int stages) {
  constexpr int kES = (int)sizeof(T);
  constexpr int kCW = 32 / TL, kCh = kWarps * kCW, kTT = TL * TS;
  constexpr int kChBytes = kCh * kES;                      // of one row of u, dt, z
  constexpr int kPiece = kChBytes < 16 ? kChBytes : 16;    // 8 bytes where a row has no more
  constexpr int kPieces = kChBytes / kPiece;
  extern __shared__ __align__(128) uint8_t smem[];
  const Layout<kES, TL, TS> lay(p.N, stages);
  float* spread_b = reinterpret_cast<float*>(smem + lay.spread);  // [N][kTT + 4]
  float* spread_c = spread_b + p.N * (kTT + 4);
  int* tokens = reinterpret_cast<int*>(smem + lay.tokens);        // [3][kTT]: next, this, last tile
  float* a_table = reinterpret_cast<float*>(smem + lay.table);    // [N][kCh]: A log2(e)
  float* carry = a_table + p.N * kCh;                             // [N][kCh]: h so far

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int tl = lane % TL, cw = lane / TL;
  const int c = warp * kCW + cw;  // channel within the CTA
  const int d0 = blockIdx.x * kCh, b = blockIdx.y;
  const int g = d0 / (p.D / p.G);

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");

  const int len = p.lengths ? min(max(__ldg(p.lengths + b), 0), p.L) : p.L;
  const int tiles = (len + kTT - 1) / kTT;
  for (int i = tid; i < p.N * kCh; i += kThreads) {
    const int ch = i / p.N, n = i - ch * p.N;
    a_table[n * kCh + ch] = __ldg(p.A + (long long)(d0 + ch) * p.N + n) * kLog2e;
    carry[n * kCh + ch] = p.state_in ? p.state_in[((long long)b * p.D + d0 + ch) * p.N + n] : 0.f;
  }
  const float skip = p.skip ? __ldg(p.skip + d0 + c) : 0.f;
  const float bias = p.dt_bias ? __ldg(p.dt_bias + d0 + c) : 0.f;

  const auto set_tokens = [&](int tile) {
    for (int r = tid; r < kTT; r += kThreads) {
      const int s = tile * kTT + r;
      tokens[(tile % 3) * kTT + r] = s < len ? p.map.token((unsigned)s) : -1;
    }
  };
  const long long row0 = (long long)b * p.L;
  const auto load_tile = [&](int tile) {
    uint8_t* st = smem + (stages == 2 ? (tile & 1) * lay.stage : 0);
    const int* tok = tokens + (tile % 3) * kTT;
    for (int i = tid; i < kTT * kPieces; i += kThreads) {
      const int r = i / kPieces, q = i - r * kPieces;
      const int m = tok[r];
      const long long row = row0 + max(m, 0);
      const int off = (r / TS) * lay.ch_block + (r % TS) * kChBytes + q * kPiece;
      const int e = d0 + q * (kPiece / kES);
      copy_async<kPiece>(st + off, static_cast<const T*>(p.u) + row * p.u_ld + e, m >= 0);
      copy_async<kPiece>(st + lay.ch_tile + off, static_cast<const T*>(p.dt) + row * p.dt_ld + e, m >= 0);
      if (p.z) copy_async<kPiece>(st + 2 * lay.ch_tile + off, static_cast<const T*>(p.z) + row * p.z_ld + e, m >= 0);
    }
    const int np = p.N * kES / 16;
    for (int i = tid; i < kTT * np; i += kThreads) {
      const int r = i / np, q = i - r * np;
      const int m = tok[r];
      const long long row = row0 + max(m, 0);
      const int off = 3 * lay.ch_tile + (r / TS) * lay.n_block + (r % TS) * p.N * kES + q * 16;
      const int e = g * p.N + q * (16 / kES);
      copy_async<16>(st + off, static_cast<const T*>(p.Bm) + row * p.bm_ld + e, m >= 0);
      copy_async<16>(st + lay.n_tile + off, static_cast<const T*>(p.Cm) + row * p.cm_ld + e, m >= 0);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  if (tiles > 0) {
    set_tokens(0);
    __syncthreads();
    load_tile(0);
  }
  for (int tile = 0; tile < tiles; ++tile) {
    const bool more = tile + 1 < tiles;
    uint8_t* st = smem + (stages == 2 ? (tile & 1) * lay.stage : 0);
    if (more) set_tokens(tile + 1);
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();  // this tile is here; the other stage's outputs have left; tokens are set
    if (stages == 2 && more) load_tile(tile + 1);

    // B and C as fp32, state by state in the order of the lanes' 16-byte reads: position
    // t = l TS + 4 q + r of the tile at (q TL + l) 4 + r
    {
      const int np = p.N * kES / 16;
      for (int i = tid; i < kTT * np; i += kThreads) {
        const int piece = i / kTT, k = i - piece * kTT;  // k: place in that order
        const int r = ((k / 4) % TL) * TS + (k / (4 * TL)) * 4 + k % 4;
        const uint8_t* src = st + 3 * lay.ch_tile + (r / TS) * lay.n_block + (r % TS) * p.N * kES + piece * 16;
        float f[16 / kES], h[16 / kES];
        Vec8<T>::load(*reinterpret_cast<const uint4*>(src), f);
        Vec8<T>::load(*reinterpret_cast<const uint4*>(src + lay.n_tile), h);
#pragma unroll
        for (int e = 0; e < 16 / kES; ++e) {
          spread_b[(piece * (16 / kES) + e) * (kTT + 4) + k] = f[e];
          spread_c[(piece * (16 / kES) + e) * (kTT + 4) + k] = h[e];
        }
      }
    }
    // this lane's positions
    float dl[TS], du[TS], y[TS], sum = 0.f;
    T* up = reinterpret_cast<T*>(st + tl * lay.ch_block) + c;
    const T* dp = reinterpret_cast<const T*>(st + lay.ch_tile + tl * lay.ch_block) + c;
    const int left = len - tile * kTT - tl * TS;  // positions of the sequence from here on
#pragma unroll
    for (int i = 0; i < TS; ++i) {
      const float u = Elem<T>::to_f32(up[i * kCh]);
      float x = Elem<T>::to_f32(dp[i * kCh]) + bias;
      if (p.softplus) x = softplus_f32(x);
      dl[i] = i < left ? x : 0.f;
      du[i] = dl[i] * u;
      y[i] = skip * u;
      sum += dl[i];
    }
    __syncthreads();  // B and C are spread

    for (int n0 = 0; n0 < p.N; n0 += NU) {
      float a[NU][TS], bb[NU][TS], h[NU], P[NU], in[NU];
#pragma unroll
      for (int v = 0; v < NU; ++v) {
        const float A = a_table[(n0 + v) * kCh + c];
        in[v] = carry[(n0 + v) * kCh + c];
        const float4* bp = reinterpret_cast<const float4*>(spread_b + (n0 + v) * (kTT + 4)) + tl;
        P[v] = exp2_approx(sum * A);
        h[v] = 0.f;
#pragma unroll
        for (int q = 0; q < TS / 4; ++q) {
          const float4 f = bp[q * TL];
          bb[v][4 * q] = du[4 * q] * f.x;
          bb[v][4 * q + 1] = du[4 * q + 1] * f.y;
          bb[v][4 * q + 2] = du[4 * q + 2] * f.z;
          bb[v][4 * q + 3] = du[4 * q + 3] * f.w;
        }
#pragma unroll
        for (int i = 0; i < TS; ++i) a[v][i] = exp2_approx(dl[i] * A);
#pragma unroll
        for (int i = 0; i < TS; ++i) h[v] = fmaf(a[v][i], h[v], bb[v][i]);
        if (tl == 0) h[v] = fmaf(P[v], in[v], h[v]);
      }
      __syncwarp();  // every lane has the old carry
#pragma unroll
      for (int s = 1; s < TL; s *= 2) {
#pragma unroll
        for (int v = 0; v < NU; ++v) {
          const float hp = __shfl_up_sync(0xffffffffu, h[v], s, TL);
          if (tl >= s) h[v] = fmaf(P[v], hp, h[v]);
          if (2 * s < TL) {
            const float Pp = __shfl_up_sync(0xffffffffu, P[v], s, TL);
            if (tl >= s) P[v] *= Pp;
          }
        }
      }
#pragma unroll
      for (int v = 0; v < NU; ++v) {
        const float hp = __shfl_up_sync(0xffffffffu, h[v], 1, TL);
        if (tl > 0) in[v] = hp;
        const float4* cp = reinterpret_cast<const float4*>(spread_c + (n0 + v) * (kTT + 4)) + tl;
#pragma unroll
        for (int q = 0; q < TS / 4; ++q) {
          const float4 f = cp[q * TL];
          in[v] = fmaf(a[v][4 * q], in[v], bb[v][4 * q]);
          y[4 * q] = fmaf(f.x, in[v], y[4 * q]);
          in[v] = fmaf(a[v][4 * q + 1], in[v], bb[v][4 * q + 1]);
          y[4 * q + 1] = fmaf(f.y, in[v], y[4 * q + 1]);
          in[v] = fmaf(a[v][4 * q + 2], in[v], bb[v][4 * q + 2]);
          y[4 * q + 2] = fmaf(f.z, in[v], y[4 * q + 2]);
          in[v] = fmaf(a[v][4 * q + 3], in[v], bb[v][4 * q + 3]);
          y[4 * q + 3] = fmaf(f.w, in[v], y[4 * q + 3]);
        }
        if (tl == TL - 1) carry[(n0 + v) * kCh + c] = in[v];
      }
    }
    const T* zp = reinterpret_cast<const T*>(st + 2 * lay.ch_tile + tl * lay.ch_block) + c;
#pragma unroll
    for (int i = 0; i < TS; ++i) {
      if (p.z) y[i] *= ssm_silu(Elem<T>::to_f32(zp[i * kCh]));
      up[i * kCh] = Elem<T>::from_f32(y[i]);
    }
    __syncthreads();  // outputs are in the place of u; the spread B and C have been read
    {
      const int* tok = tokens + (tile % 3) * kTT;
      for (int i = tid; i < kTT * kPieces; i += kThreads) {
        const int r = i / kPieces, q = i - r * kPieces;
        const int m = tok[r];
        if (m < 0) continue;
        const uint8_t* src = st + (r / TS) * lay.ch_block + (r % TS) * kChBytes + q * kPiece;
        T* dst = static_cast<T*>(p.out) + (row0 + m) * p.D + d0 + q * (kPiece / kES);
        if constexpr (kPiece == 16)
          *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(src);
        else
          *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<const uint2*>(src);
      }
    }
    if (stages == 1 && more) {
      __syncthreads();  // the stage is free
      load_tile(tile + 1);
    }
  }
  if (p.state_out) {
    __syncthreads();
    for (int i = tid; i < p.N * kCh; i += kThreads) {
      const int ch = i / p.N, n = i - ch * p.N;
      p.state_out[((long long)b * p.D + d0 + ch) * p.N + n] = carry[n * kCh + ch];
    }
  }
}

constexpr int kMaxSmem = 227 * 1024;

template <typename T, int TL, int TS, int NU>
gtr_status_t launch_scan(const SsmParams& p, int stages, cudaStream_t stream) {
  static std::once_flag once;
  static cudaError_t attr = cudaSuccess;
  std::call_once(once, [] {
    attr = cudaFuncSetAttribute(ssm_scan_kernel<T, TL, TS, NU>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
  });
  if (attr != cudaSuccess) return GTR_ERR_CUDA;
  constexpr int kCh = kWarps * 32 / TL;
  const Layout<(int)sizeof(T), TL, TS> lay(p.N, stages);
  return launch_serial(ssm_scan_kernel<T, TL, TS, NU>, dim3((unsigned)(p.D / kCh), (unsigned)p.B), dim3(kThreads),
                       (size_t)lay.total, stream, p, stages);
}

template <typename T>
gtr_status_t launch_scan_t(const SsmParams& p, cudaStream_t stream) {
  constexpr int es = (int)sizeof(T);
  const int tiles16 = p.B * (p.D / 16);
  if (tiles16 < 148 && Layout<es, 32, 8>(p.N, 1).total <= kMaxSmem) {
    const int stages = Layout<es, 32, 8>(p.N, 2).total <= kMaxSmem / 2 ? 2 : 1;
    return launch_scan<T, 32, 8, 4>(p, stages, stream);
  }
  const int stages = Layout<es, 8, 16>(p.N, 2).total <= kMaxSmem / 3 ? 2 : 1;
  return launch_scan<T, 8, 16, 1>(p, stages, stream);
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
  switch (dtype) {
    case GTR_F16: return launch_scan_t<__half>(p, s);
    case GTR_BF16: return launch_scan_t<__nv_bfloat16>(p, s);
    default: return launch_scan_t<float>(p, s);
  }
}
