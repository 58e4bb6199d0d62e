// The norms around a block, fused with the block's gate, its residual scale and the residual
// stream.  Per token row (C channels), y the block's output and h the residual stream:
//
//     p  = y / sqrt(mean_c y^2 + eps) * post_w        (no post_w: p = y)
//     h' = h + scale * act(gate) * p                  (no scale, no gate: factor 1)
//     n  = h' / sqrt(mean_c h'^2 + eps) * pre_w       (from h' before its rounding)
//
// One pass over the data: a row is held in the registers of TPR threads (a warp for short rows,
// a block above), one or two 16-byte pieces each, the two sums of squares are reduced in fp32
// with shuffles and one barrier each, and h' never returns from memory for its norm.
//
// Bound by HBM bandwidth: y, h and the gate are read once, h' and n written once.  What keeps
// loads in flight is the number of resident rows, so a thread holds little: requesting the
// weights of the second half early, or walking over rows with weights and the next row in
// registers, measured 20 to 60% slower on large inputs.  Measured: 30,720 rows of 1536, bf16
// with fp32 residual, 98 us, 88% of the measured HBM bandwidth; 1600 rows of 384, fp16, 3.0 us.
// Rows above 4096 leave one or two blocks on an SM, whose loads, sums and stores follow one
// another: bf16 with a gate for each token, 2441 rows of 8192 51 us, 60%; 1220 of 16384 78 us, 39%.
#include "gtr_common.cuh"
#include "gtr_launch.cuh"
#include "gtr_math.cuh"
#include "gtr_vec.cuh"

namespace gtr {
namespace {

struct NormParams {
  const void* y;
  const void* h;
  const float* post_w;  // [C] or nullptr
  const float* pre_w;   // [C] or nullptr (then n is not written)
  const void* gate;     // [B][C] or [B][L][C] or nullptr
  const float* scale;   // [C] or nullptr
  void* h_out;
  void* n_out;
  float eps;
  long long rows;
  int L, C, gate_rows, silu;  // gate_rows: 0 none, 1 per sequence, 2 per token
};

// N consecutive values of T as fp32, N a multiple of 16 / sizeof(T)
template <typename T, int N>
__device__ __forceinline__ void load_row(const T* p, float* f) {
#pragma unroll
  for (int i = 0; i < N; i += Vec8<T>::N) {
    const uint4 u = *reinterpret_cast<const uint4*>(p + i);
    Vec8<T>::load(u, f + i);
  }
}
template <typename T, int N>
__device__ __forceinline__ void store_row(T* p, const float* f) {
#pragma unroll
  for (int i = 0; i < N; i += Vec8<T>::N) __stcs(reinterpret_cast<uint4*>(p + i), Vec8<T>::store(f + i));
}

// Sum over the row's TPR threads, the same value in each of them.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (TPR > 32) {
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < TPR / 32; ++i) v += red[i];
  }
  return v;
}

// T: y, gate and n; R: the residual stream; NV pieces of 16 / sizeof(T) channels a thread.
template <typename T, typename R, int TPR, int NV>
__global__ void __launch_bounds__(TPR == 32 ? 128 : TPR) block_norm_kernel(const NormParams p) {
  constexpr int kN = Vec8<T>::N;
  constexpr int kRowsPerCta = TPR == 32 ? 4 : 1;
  __shared__ float red[2][TPR / 32];  // one buffer for each sum: one barrier each
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x % TPR;
  const long long row = (long long)blockIdx.x * kRowsPerCta + threadIdx.x / TPR;
  if (row >= p.rows) return;  // whole rows' threads at once: they are whole warps, or the CTA
  const int nvec = p.C / kN;
  const T* y = static_cast<const T*>(p.y) + row * p.C;
  const R* h = static_cast<const R*>(p.h) + row * p.C;
  const T* gate = static_cast<const T*>(p.gate) + (p.gate_rows == 1 ? row / p.L : row) * p.C;
  float fy[NV][kN], fh[NV][kN];
  uint4 fg[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = (v * TPR + lane) * kN;
#pragma unroll
    for (int e = 0; e < kN; ++e) fy[v][e] = fh[v][e] = 0.f;
    fg[v] = make_uint4(0, 0, 0, 0);
    if (v * TPR + lane < nvec) {
      load_row<T, kN>(y + c, fy[v]);
      load_row<R, kN>(h + c, fh[v]);
      if (p.gate_rows) fg[v] = *reinterpret_cast<const uint4*>(gate + c);
    }
  }
  float rp = 1.f;
  if (p.post_w) {
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < kN; ++e) s = fmaf(fy[v][e], fy[v][e], s);
    rp = rsqrtf(row_sum<TPR>(s, red[0]) / (float)p.C + p.eps);
  }
  float s2 = 0.f;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = (v * TPR + lane) * kN;
    if (v * TPR + lane < nvec) {
      float f[kN];
      if (p.post_w) {
        load_row<float, kN>(p.post_w + c, f);
#pragma unroll
        for (int e = 0; e < kN; ++e) fy[v][e] *= rp * f[e];
      }
      if (p.gate_rows) {
        Vec8<T>::load(fg[v], f);
#pragma unroll
        for (int e = 0; e < kN; ++e) fy[v][e] *= p.silu ? silu_f32(f[e]) : f[e];
      }
      if (p.scale) {
        load_row<float, kN>(p.scale + c, f);
#pragma unroll
        for (int e = 0; e < kN; ++e) fy[v][e] *= f[e];
      }
#pragma unroll
      for (int e = 0; e < kN; ++e) {
        fh[v][e] += fy[v][e];
        s2 = fmaf(fh[v][e], fh[v][e], s2);
      }
      store_row<R, kN>(static_cast<R*>(p.h_out) + row * p.C + c, fh[v]);
    }
  }
  if (!p.pre_w) return;
  const float rn = rsqrtf(row_sum<TPR>(s2, red[1]) / (float)p.C + p.eps);
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = (v * TPR + lane) * kN;
    if (v * TPR + lane < nvec) {
      float f[kN];
      load_row<float, kN>(p.pre_w + c, f);
#pragma unroll
      for (int e = 0; e < kN; ++e) f[e] *= rn * fh[v][e];
      store_row<T, kN>(static_cast<T*>(p.n_out) + row * p.C + c, f);
    }
  }
}

template <typename T, typename R, int TPR, int NV>
gtr_status_t launch_norm(const NormParams& p, cudaStream_t stream) {
  constexpr int kRowsPerCta = TPR == 32 ? 4 : 1;
  const long long grid = (p.rows + kRowsPerCta - 1) / kRowsPerCta;
  if (grid > 0x7fffffffll) return GTR_ERR_UNSUPPORTED;
  return launch_serial(block_norm_kernel<T, R, TPR, NV>, dim3((unsigned)grid), dim3(TPR == 32 ? 128 : TPR), 0, stream, p);
}

// TPR by the row's pieces.  Up to 64 pieces a warp holds two a thread, except where the rows are
// few: two warps a row with one piece a thread are quicker (1600 rows of 384, fp16: 2.95 us, a
// warp 3.44 us).  They are for many rows as well (54,000 rows, bf16: 43 us, a warp 47 us), which
// this rule does not use.  Up to 256 pieces one a thread (30,720 rows of 192 pieces: 98 us, two a
// thread 100 us); above, two: a block of half the threads waits less at its barriers.
template <typename T, typename R>
gtr_status_t launch_norm_c(const NormParams& p, cudaStream_t stream) {
  const int nvec = p.C / Vec8<T>::N;
  if (nvec <= 32) return launch_norm<T, R, 32, 1>(p, stream);
  if (nvec <= 64) return p.rows <= 148 * 16 ? launch_norm<T, R, 64, 1>(p, stream) : launch_norm<T, R, 32, 2>(p, stream);
  if (nvec <= 96) return launch_norm<T, R, 96, 1>(p, stream);
  if (nvec <= 128) return launch_norm<T, R, 128, 1>(p, stream);
  if (nvec <= 192) return launch_norm<T, R, 192, 1>(p, stream);
  if (nvec <= 256) return launch_norm<T, R, 256, 1>(p, stream);
  if (nvec <= 320) return launch_norm<T, R, 160, 2>(p, stream);
  if (nvec <= 384) return launch_norm<T, R, 192, 2>(p, stream);
  if (nvec <= 512) return launch_norm<T, R, 256, 2>(p, stream);
  if (nvec <= 1024) return launch_norm<T, R, 512, 2>(p, stream);
  return launch_norm<T, R, 512, 4>(p, stream);
}

}  // namespace
}  // namespace gtr

extern "C" gtr_status_t gtr_block_norm(const void* y, const void* h, const float* post_w, const float* pre_w,
                                       const void* gate, int gate_per_token, int gate_silu, const float* scale,
                                       float eps, void* h_out, void* n_out, int B, int64_t L, int C, int dtype,
                                       int residual_dtype, gtr_stream_t stream) {
  using namespace gtr;
  if (!y || !h || !h_out || (pre_w != nullptr) != (n_out != nullptr) || B <= 0 || L <= 0 || C <= 0)
    return GTR_ERR_INVALID_ARG;
  if (dtype < GTR_F32 || dtype > GTR_BF16 || residual_dtype < GTR_F32 || residual_dtype > GTR_BF16)
    return GTR_ERR_INVALID_ARG;
  if (!(eps >= 0.f) || eps > 3.4e38f) return GTR_ERR_INVALID_ARG;
  for (const void* q : {y, h, (const void*)post_w, (const void*)pre_w, gate, (const void*)scale, (const void*)h_out,
                        (const void*)n_out})
    if (!aligned_to(q, 16)) return GTR_ERR_INVALID_ARG;
  if (residual_dtype != dtype && residual_dtype != GTR_F32) return GTR_ERR_UNSUPPORTED;
  const int es = dtype == GTR_F32 ? 4 : 2, er = residual_dtype == GTR_F32 ? 4 : 2;
  if (C % (16 / es) != 0 || C > 2048 * (16 / es)) return GTR_ERR_UNSUPPORTED;
  if (L > (1ll << 28) || (double)B * L * C >= 1e12) return GTR_ERR_UNSUPPORTED;
  const long long rows = (long long)B * L;
  const size_t ny = (size_t)rows * C * es, nh = (size_t)rows * C * er, nw = (size_t)C * 4;
  const size_t ng = (size_t)(gate_per_token ? rows : B) * C * es;
  if ((h_out != h && overlaps(h_out, nh, h, nh)) || overlaps(h_out, nh, y, ny) || overlaps(h_out, nh, gate, ng) ||
      overlaps(h_out, nh, n_out, ny) || overlaps(n_out, ny, h, nh) || (n_out != y && overlaps(n_out, ny, y, ny)) ||
      overlaps(n_out, ny, gate, ng))
    return GTR_ERR_INVALID_ARG;
  for (const void* q : {post_w, pre_w, scale})
    if (overlaps(h_out, nh, q, nw) || overlaps(n_out, ny, q, nw)) return GTR_ERR_INVALID_ARG;
  NormParams p{y, h, post_w, pre_w, gate, scale, h_out, n_out, eps, rows, (int)L, C,
               gate ? (gate_per_token ? 2 : 1) : 0, gate_silu != 0};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool wide = residual_dtype == GTR_F32;
  switch (dtype) {
    case GTR_F16: return wide ? launch_norm_c<__half, float>(p, s) : launch_norm_c<__half, __half>(p, s);
    case GTR_BF16:
      return wide ? launch_norm_c<__nv_bfloat16, float>(p, s) : launch_norm_c<__nv_bfloat16, __nv_bfloat16>(p, s);
    default: return launch_norm_c<float, float>(p, s);
  }
}
