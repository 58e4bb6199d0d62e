// Short causal depthwise convolution along the scan, with carried inputs and SiLU.
//
//     out_s[c] = act( bias[c] + sum_{k < K} w[c, k] x_{s - K + 1 + k}[c] ),   K = 2, 3 or 4,
//
// s the position in the scan order; positions before the first are the carried inputs (or
// zero), and the sequence's last K - 1 inputs are carried on.
//
// A thread owns one 16-byte piece of the channels (8 of 16-bit data, 4 of fp32) and a strip of
// consecutive positions; its taps are registers and it slides along, the next rows on their
// way.  Neighbouring threads hold neighbouring pieces, so a warp reads and writes whole rows
// whatever the direction: the direction only changes which row comes next.
//
// Bound: HBM, 2 elements of traffic for 2 K + 5 operations.  Measured (bf16, K = 4, SiLU): eight
// 48 x 80 grids of 1152 channels 32 us, 67% of the measured HBM bandwidth (K = 2 29 us, 76%; fp32
// 48 us, 90%); one 128 x 128 grid of 768 channels 16 us, 48% (fp32 21 us, 75%): a few blocks more
// than a wave, see launch_conv; one 40 x 40 grid of 768 channels 4.0 us.  It was 54 us on the first
// and 12 us on the last with taps read from global memory by each thread and strips of 8 and 4
// positions.
#include "gtr_common.cuh"
#include "gtr_launch.cuh"
#include "gtr_math.cuh"
#include "gtr_scan_order.cuh"
#include "gtr_sm100.cuh"
#include "gtr_vec.cuh"

namespace gtr {
namespace {

constexpr int kConvThreads = 128;
constexpr int kDepth = 8;

struct ConvParams {
  const void* x;
  long long x_ld;
  const float* w;     // [C][K]
  const float* bias;  // [C] or nullptr
  const void* state_in;  // [B][K-1][C] or nullptr
  void* state_out;       // [B][K-1][C] or nullptr; may be state_in
  const int* lengths;    // [B] or nullptr
  void* out;
  int B, L, C, silu, strip;
  unsigned nvec, strips, total;  // pieces per row, strips per sequence, threads with work
  ScanMap map;
};

// A strip of p.strip positions.  Its rows wait in a ring of kDepth slots in shared memory, which
// each thread fills (cp.async) and reads for itself: that many rows are on their way per
// thread without a register held for them, and no thread waits for another.
template <typename T, int K>
__global__ void __launch_bounds__(kConvThreads) ssm_conv_kernel(const ConvParams p) {
  constexpr int kN = Vec8<T>::N;
  __shared__ uint4 ring[kDepth][kConvThreads];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const unsigned idx = blockIdx.x * (unsigned)kConvThreads + threadIdx.x;
  const unsigned row = idx / p.nvec, vec = idx - row * p.nvec;
  const unsigned b = min(row / p.strips, (unsigned)p.B - 1), strip = row - b * p.strips;
  const int s0 = (int)strip * p.strip;
  const int len = p.lengths ? min(max(__ldg(p.lengths + b), 0), p.L) : p.L;
  const bool has_work = idx < p.total && (strip == 0 || s0 < len);
  if (!__any_sync(0xffffffffu, has_work)) return;
  const int s1 = has_work ? min(s0 + p.strip, len) : s0;

  const int c0 = (int)vec * kN;
  const T* x = static_cast<const T*>(p.x) + (long long)b * p.L * p.x_ld + c0;
  const T* state_in = p.state_in ? static_cast<const T*>(p.state_in) + (long long)b * (K - 1) * p.C + c0 : nullptr;
  const auto row_of = [&](int token) { return reinterpret_cast<const uint4*>(x + (long long)token * p.x_ld); };

  ScanWalk at(p.map, (unsigned)s0);  // the next row to request
  const uint32_t slot0 = sm100::smem_u32(&ring[0][threadIdx.x]);
  const auto request = [&](int s, int slot) {  // row s of the strip's, if it has one; one group either way
    if (s < s1) {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(slot0 + slot * (kConvThreads * 16)),
                   "l"(row_of(at.token))
                   : "memory");
      at.next(p.map);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kDepth; ++i) request(s0 + i, i);

  // the K - 1 rows before the strip; before position 0 the carried inputs.  They are read
  // before state_out (which may be the same buffer) is written: the thread of a sequence's
  // first strip is the only one that touches its piece of either (a strip has at least K - 1
  // positions wherever there is a second one)
  uint4 before[K - 1];
#pragma unroll
  for (int j = 0; j < K - 1; ++j) {
    before[j] = make_uint4(0, 0, 0, 0);
    if (has_work && strip != 0)
      before[j] = __ldg(row_of(p.map.token((unsigned)(s0 - K + 1 + j))));
    else if (has_work && state_in)
      before[j] = *reinterpret_cast<const uint4*>(state_in + (long long)j * p.C);
  }

  // The warp's taps, kN K floats a lane, by whole lines into shared memory and from there to
  // each lane: read directly, every lane's 16 bytes would be a line of their own, as costly as
  // two dozen rows of the strip.  The lanes' pieces follow one another, from the last of a row
  // to the first of the next.
  constexpr int kTaps = kN * K, kQuads = kTaps / 4;
  constexpr int kTapStride = kTaps + (kQuads % 2 ? 8 : 4);  // an odd number of 16-byte pieces
  __shared__ float4 tap_smem[kConvThreads / 32][32 * kTapStride / 4];
  float* taps = reinterpret_cast<float*>(tap_smem[threadIdx.x / 32]);
  const unsigned vec0 = __shfl_sync(0xffffffffu, vec, 0);
#pragma unroll
  for (int i = 0; i < kQuads; ++i) {
    const unsigned k = i * 32 + threadIdx.x % 32, l = k / kQuads, o = k % kQuads;
    unsigned v = vec0 + l;
    if (v >= p.nvec) v %= p.nvec;
    *reinterpret_cast<float4*>(taps + l * kTapStride + o * 4) =
        __ldg(reinterpret_cast<const float4*>(p.w + (size_t)v * kTaps) + o);
  }
  __syncwarp();
  if (!has_work) return;

  float2 f[K][kN / 2];  // the window, oldest first
#pragma unroll
  for (int j = 0; j < K - 1; ++j) Vec8<T>::load(before[j], &f[j + 1][0].x);
  float2 w[K][kN / 2], bias[kN / 2];
  {
    float v[kTaps];
#pragma unroll
    for (int i = 0; i < kQuads; ++i) {
      const float4 q = *reinterpret_cast<const float4*>(taps + threadIdx.x % 32 * kTapStride + i * 4);
      v[4 * i] = q.x, v[4 * i + 1] = q.y, v[4 * i + 2] = q.z, v[4 * i + 3] = q.w;
    }
#pragma unroll
    for (int e = 0; e < kN / 2; ++e)
#pragma unroll
      for (int k = 0; k < K; ++k) w[k][e] = make_float2(v[2 * e * K + k], v[(2 * e + 1) * K + k]);
  }
#pragma unroll
  for (int e = 0; e < kN; e += 4) {
    const float4 v = p.bias ? __ldg(reinterpret_cast<const float4*>(p.bias + c0 + e)) : make_float4(0.f, 0.f, 0.f, 0.f);
    bias[e / 2] = make_float2(v.x, v.y), bias[e / 2 + 1] = make_float2(v.z, v.w);
  }
  T* out = static_cast<T*>(p.out) + (long long)b * p.L * p.C + c0;
  ScanWalk to(p.map, (unsigned)s0);
  int slot = 0;
#pragma unroll K
  for (int s = s0; s < s1; ++s) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
    const uint4 r = ring[slot][threadIdx.x];
#pragma unroll
    for (int j = 0; j < K - 1; ++j)
#pragma unroll
      for (int e = 0; e < kN / 2; ++e) f[j][e] = f[j + 1][e];
    Vec8<T>::load(r, &f[K - 1][0].x);
    request(s + kDepth, slot);  // the slot has been read
    slot = slot + 1 == kDepth ? 0 : slot + 1;
    float2 y[kN / 2];
#pragma unroll
    for (int e = 0; e < kN / 2; ++e) {
      y[e] = bias[e];
#pragma unroll
      for (int k = 0; k < K; ++k) y[e] = fma2(w[k][e], f[k][e], y[e]);
    }
    if (p.silu) {
#pragma unroll
      for (int e = 0; e < kN / 2; ++e) y[e] = silu2(y[e]);
    }
    *reinterpret_cast<uint4*>(out + (long long)to.token * p.C) = Vec8<T>::store(&y[0].x);
    to.next(p.map);
  }
  if (strip == 0 && p.state_out) {
    T* state_out = static_cast<T*>(p.state_out) + (long long)b * (K - 1) * p.C + c0;
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      uint4 keep;
      if (len <= p.strip) {  // the window's end is the sequence's; its values are x's own
        keep = Vec8<T>::store(&f[j + 1][0].x);
      } else {
        keep = __ldg(row_of(p.map.token((unsigned)(len - (K - 1) + j))));
      }
      *reinterpret_cast<uint4*>(state_out + (long long)j * p.C) = keep;
    }
  }
}

template <typename T, int K>
gtr_status_t launch_conv(ConvParams p, int B, cudaStream_t stream) {
  p.nvec = (unsigned)(p.C / Vec8<T>::N);
  // A strip is about as long as makes one wave of four blocks an SM, 4 to 24 positions: a shorter
  // one pays its taps and its K - 1 rows too often (eight 48 x 80 grids of 1152 channels, bf16: 4
  // positions 51 us, 24 32 us), a longer one leaves SMs idle (one 40 x 40 grid of 768 channels: 4
  // positions 4.0 us, 24 6.4 us).  Four blocks is what 16-bit data and K = 3 or 4 hold (102 and 124
  // registers); the other kernels hold six to eight.  The share is cut to whole positions first,
  // so a launch may have a few blocks more than the wave (one 128 x 128 grid of 768 channels: 615
  // for 592, 16.0 us; strips of 28 13.6 us).
  const long long fair = (long long)B * p.L * p.nvec / (4ll * 148 * kConvThreads);
  p.strip = p.L == 1 ? 1 : (int)(fair < 4 ? 4 : fair > 24 ? 24 : (fair + 3) / 4 * 4);
  p.strips = (unsigned)((p.L + p.strip - 1) / p.strip);
  const unsigned long long total = (unsigned long long)B * p.strips * p.nvec;
  if (total >= 1ull << 32) return GTR_ERR_UNSUPPORTED;
  p.total = (unsigned)total;
  const dim3 grid((unsigned)((total + kConvThreads - 1) / kConvThreads));
  return launch_serial(ssm_conv_kernel<T, K>, grid, dim3(kConvThreads), 0, stream, p);
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
  if (!aligned_to(x, 16) || !aligned_to(out, 16) || !aligned_to(w, 16) || !aligned_to(bias, 16) ||
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
  const struct {
    const void* q;
    size_t n;
  } params[] = {{w, (size_t)C * K * 4}, {bias, (size_t)C * 4}, {lengths, (size_t)B * 4}};
  for (const auto& i : params)
    if (overlaps(out, no, i.q, i.n) || overlaps(state_out, ns, i.q, i.n)) return GTR_ERR_INVALID_ARG;
  ConvParams p{x, x_ld, w, bias, state_in, state_out, lengths, out, B, (int)L, C, silu != 0, 0, 0, 0, 0,
               ScanMap::make(direction, grid_H, grid_W)};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  switch (dtype) {
    case GTR_F16: return launch_conv_k<__half>(p, B, K, s);
    case GTR_BF16: return launch_conv_k<__nv_bfloat16>(p, B, K, s);
    default: return launch_conv_k<float>(p, B, K, s);
  }
}
