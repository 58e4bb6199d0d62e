// Short causal depthwise convolution along the scan, with carried inputs and SiLU.
//
//     out_s[c] = act( bias[c] + sum_{k < K} w[c, k] x_{s - K + 1 + k}[c] ),   K = 2, 3 or 4,
//
// s the position in the scan order; positions before the first are the carried inputs (or
// zero), and the sequence's last K - 1 inputs are carried on.
//
// A thread owns one 16-byte piece of the channels (8 of 16-bit data, 4 of fp32) and a strip
// of S consecutive positions: it requests the strip's S + K - 1 rows at once (the K - 1 rows
// before the strip were a neighbour's, and come from L2), keeps its taps in registers and
// slides along.  Neighbouring threads hold neighbouring pieces, so a warp reads and writes
// whole rows whatever the direction: the direction only changes which row comes next.  The
// convolution is bound by HBM bandwidth: 2 elements of traffic for 2 K + 5 operations.
#include "gtr_common.cuh"
#include "gtr_launch.cuh"
#include "gtr_scan_order.cuh"
#include "gtr_vec.cuh"

namespace gtr {
namespace {

constexpr int kConvThreads = 128;

struct ConvParams {
  const void* x;
  long long x_ld;
  const float* w;     // [C][K]
  const float* bias;  // [C] or nullptr
  const void* state_in;  // [B][K-1][C] or nullptr
  void* state_out;       // [B][K-1][C] or nullptr; may be state_in
  const int* lengths;    // [B] or nullptr
  void* out;
  int L, C, silu;
  unsigned nvec, strips, total;  // pieces per row, strips per sequence, threads with work
  ScanMap map;
};

__device__ __forceinline__ float silu_f32(float x) { return __fdividef(x, 1.f + __expf(-x)); }

template <typename T, int K, int S>
__global__ void __launch_bounds__(kConvThreads) ssm_conv_kernel(const ConvParams p) {
  constexpr int kN = Vec8<T>::N;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const unsigned idx = blockIdx.x * (unsigned)kConvThreads + threadIdx.x;
  if (idx >= p.total) return;
  const unsigned row = idx / p.nvec, vec = idx - row * p.nvec;
  const unsigned b = row / p.strips, strip = row - b * p.strips;
  const int s0 = (int)strip * S;
  const int len = p.lengths ? min(max(__ldg(p.lengths + b), 0), p.L) : p.L;
  if (strip != 0 && s0 >= len) return;

  const int c0 = (int)vec * kN;
  const T* x = static_cast<const T*>(p.x) + (long long)b * p.L * p.x_ld + c0;
  // the carried inputs, read before state_out (which may be the same buffer) is written:
  // the thread of a sequence's first strip is the only one that touches its piece of either
  uint4 st[K - 1];
#pragma unroll
  for (int j = 0; j < K - 1; ++j) st[j] = make_uint4(0, 0, 0, 0);
  if (strip == 0 && p.state_in) {
#pragma unroll
    for (int j = 0; j < K - 1; ++j)
      st[j] = *reinterpret_cast<const uint4*>(static_cast<const T*>(p.state_in) + ((long long)b * (K - 1) + j) * p.C + c0);
  }
  // rows s0 - K + 1 .. s0 + S - 1; only the first strip has rows before position 0 (S >= K - 1
  // wherever there is a second strip)
  uint4 r[S + K - 1];
  {
    ScanWalk at(p.map, strip == 0 ? 0u : (unsigned)(s0 - K + 1));
#pragma unroll
    for (int j = 0; j < S + K - 1; ++j) {
      if (strip == 0 && j < K - 1) {
        r[j] = st[j];
        continue;
      }
      r[j] = make_uint4(0, 0, 0, 0);
      if (s0 - K + 1 + j < len) r[j] = __ldg(reinterpret_cast<const uint4*>(x + (long long)at.token * p.x_ld));
      at.next(p.map);
    }
  }
  float w[K][kN], bias[kN];
#pragma unroll
  for (int e = 0; e < kN; ++e) {
#pragma unroll
    for (int k = 0; k < K; ++k) w[k][e] = __ldg(p.w + (long long)(c0 + e) * K + k);
    bias[e] = p.bias ? __ldg(p.bias + c0 + e) : 0.f;
  }
  T* out = static_cast<T*>(p.out) + (long long)b * p.L * p.C + c0;
  {
    ScanWalk at(p.map, (unsigned)s0);
    float f[K][kN];  // the window, oldest first
#pragma unroll
    for (int j = 0; j < K - 1; ++j) Vec8<T>::load(r[j], f[j + 1]);
#pragma unroll
    for (int i = 0; i < S; ++i) {
#pragma unroll
      for (int j = 0; j < K - 1; ++j)
#pragma unroll
        for (int e = 0; e < kN; ++e) f[j][e] = f[j + 1][e];
      Vec8<T>::load(r[i + K - 1], f[K - 1]);
      float y[kN];
#pragma unroll
      for (int e = 0; e < kN; ++e) {
        y[e] = bias[e];
#pragma unroll
        for (int k = 0; k < K; ++k) y[e] = fmaf(w[k][e], f[k][e], y[e]);
        if (p.silu) y[e] = silu_f32(y[e]);
      }
      if (s0 + i < len) *reinterpret_cast<uint4*>(out + (long long)at.token * p.C) = Vec8<T>::store(y);
      at.next(p.map);
    }
  }
  if (strip == 0 && p.state_out) {
    uint4 keep[K - 1];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      const int q = len - (K - 1) + j;  // the position that is carried on
      keep[j] = make_uint4(0, 0, 0, 0);
      if (q >= 0) {
        keep[j] = __ldg(reinterpret_cast<const uint4*>(x + (long long)p.map.token((unsigned)q) * p.x_ld));
      } else {
#pragma unroll
        for (int i = 0; i < K - 1; ++i)
          if (q + K - 1 == i) keep[j] = st[i];
      }
    }
#pragma unroll
    for (int j = 0; j < K - 1; ++j)
      *reinterpret_cast<uint4*>(static_cast<T*>(p.state_out) + ((long long)b * (K - 1) + j) * p.C + c0) = keep[j];
  }
}

template <typename T, int K>
gtr_status_t launch_conv(ConvParams p, int B, cudaStream_t stream) {
  p.nvec = (unsigned)(p.C / Vec8<T>::N);
  const int S = p.L == 1 ? 1 : ((long long)B * p.L * p.nvec >= 8ll * 2 * 148 * kConvThreads ? 8 : 4);
  p.strips = (unsigned)((p.L + S - 1) / S);
  const unsigned long long total = (unsigned long long)B * p.strips * p.nvec;
  if (total >= 1ull << 32) return GTR_ERR_UNSUPPORTED;
  p.total = (unsigned)total;
  const dim3 grid((unsigned)((total + kConvThreads - 1) / kConvThreads));
  if (S == 1) return launch_serial(ssm_conv_kernel<T, K, 1>, grid, dim3(kConvThreads), 0, stream, p);
  if (S == 4) return launch_serial(ssm_conv_kernel<T, K, 4>, grid, dim3(kConvThreads), 0, stream, p);
  return launch_serial(ssm_conv_kernel<T, K, 8>, grid, dim3(kConvThreads), 0, stream, p);
}

template <typename T>
gtr_status_t launch_conv_k(const ConvParams& p, int B, int K, cudaStream_t stream) {
  switch (K) {
    case 2: return launch_conv<T, 2>(p, B, stream);
    case 3: return launch_conv<T, 3>(p, B, stream);
    default: return launch_conv<T, 4>(p, B, stream);
  }
}

}  // namespace
}  // namespace gtr

extern "C" gtr_status_t gtr_ssm_conv(const void* x, int64_t x_ld, const float* w, const float* bias,
                                     const void* state_in, void* state_out, const int* lengths, void* out, int B,
                                     int grid_H, int grid_W, int C, int K, int direction, int silu, int dtype,
                                     gtr_stream_t stream) {
  using namespace gtr;
  if (!x || !w || !out || B <= 0 || grid_H <= 0 || grid_W <= 0 || C <= 0 || K <= 0) return GTR_ERR_INVALID_ARG;
  if (direction < GTR_L2R || direction > GTR_B2T || dtype < GTR_F32 || dtype > GTR_BF16) return GTR_ERR_INVALID_ARG;
  const int es = dtype == GTR_F32 ? 4 : 2;
  if (!aligned_to(x, 16) || !aligned_to(out, 16) || !aligned_to(w, 4) || !aligned_to(bias, 4) ||
      !aligned_to(state_in, 16) || !aligned_to(state_out, 16) || !aligned_to(lengths, 4))
    return GTR_ERR_INVALID_ARG;
  if (x_ld < C || x_ld % (16 / es) != 0) return GTR_ERR_INVALID_ARG;
  const long long L = (long long)grid_H * grid_W;
  if (K < 2 || K > 4 || C % (16 / es) != 0) return GTR_ERR_UNSUPPORTED;
  if (L > (1ll << 28) || C > (1 << 20) || x_ld > (1ll << 32) || (double)B * L * x_ld >= 1e12) return GTR_ERR_UNSUPPORTED;
  const size_t nx = span_bytes(B * L, x_ld, C, es), no = span_bytes(B * L, C, C, es);
  const size_t ns = span_bytes((long long)B * (K - 1), C, C, es);
  if (overlaps(out, no, x, nx) || overlaps(out, no, state_in, ns) || overlaps(out, no, state_out, ns) ||
      overlaps(state_out, ns, x, nx) || (state_in != state_out && overlaps(state_in, ns, state_out, ns)))
    return GTR_ERR_INVALID_ARG;
  ConvParams p{x, x_ld, w, bias, state_in, state_out, lengths, out, (int)L, C, silu != 0, 0, 0, 0,
               ScanMap::make(direction, grid_H, grid_W)};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  switch (dtype) {
    case GTR_F16: return launch_conv_k<__half>(p, B, K, s);
    case GTR_BF16: return launch_conv_k<__nv_bfloat16>(p, B, K, s);
    default: return launch_conv_k<float>(p, B, K, s);
  }
}
