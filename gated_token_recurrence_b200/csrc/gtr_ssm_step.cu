// Selective state space scan of one token per sequence, from and to a stored state.
//
// The N states of a channel are spread over LPC neighbouring lanes, NV float4 each, so that a
// warp reads and writes the stored states in whole sectors.  The lanes take LPC sequences
// together: A stays in registers, lane j computes delta for sequence j and hands it round by
// shuffles, and the sums over n of the LPC sequences are reduced in one transposing pass that
// leaves sequence j's in lane j, for the skip term and the gate.
//
// Bound: HBM, the states' 8 N bytes per channel in and out against 8 bytes (16-bit data) of u,
// dt, z and out.  Measured (1536 channels): 512 sequences of N = 16, bf16 23.6 us, 69% of the
// measured HBM bandwidth, fp32 25.3 us, 68%; 64 of N = 64, bf16 11.0 us, 71%, fp32 12.2 us, 65%.
// There the loads' latency is left: a thread asks for all it needs once.
#include "gtr_launch.cuh"
#include "gtr_ssm.cuh"
#include "gtr_ssm_host.h"

namespace gtr {
namespace {

constexpr int kStepThreads = 128;
// The exponent delta A log2(e) as (2 delta) (A log2(e) / 2): the same bits, and every finite rate
// stays finite, so that a step of 0 keeps the state (0 * -inf would be a NaN).
constexpr float kHalfLog2e = 0.5f * kLog2e;

// Sums over the LPC lanes of a channel of LPC values each; lane j gets the sum of value j.
template <int LPC>
__device__ __forceinline__ float transposed_sum(float (&v)[LPC], int j) {
#pragma unroll
  for (int o = LPC / 2; o > 0; o /= 2) {
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float send = (j & o) ? v[i] : v[i + o];
      const float keep = (j & o) ? v[i + o] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
    }
  }
  return v[0];
}

// R sequences a thread: LPC, or 1 where there are few: then every lane computes delta for itself.
template <typename T, int LPC, int NV, int R>
__global__ void __launch_bounds__(kStepThreads) ssm_step_kernel(const SsmParams p) {
  static_assert(R == LPC || R == 1, "");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int j = threadIdx.x % LPC;
  const int d = blockIdx.x * (kStepThreads / LPC) + threadIdx.x / LPC;
  if (d >= p.D) return;  // whole warps: D is a multiple of 16
  const int b0 = blockIdx.y * R, g = d / (p.D / p.G);
  const long long state_row = (long long)p.D * p.N;
  const float* state_in = p.state_in + (b0 * (long long)p.D + d) * p.N + 4 * j;
  float* state_out = p.state_out + (b0 * (long long)p.D + d) * p.N + 4 * j;

  float4 h[R][NV];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      h[r][v] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (b0 + r < p.B) h[r][v] = __ldcs(reinterpret_cast<const float4*>(state_in + r * state_row + 4 * LPC * v));
    }
  const int own = R == 1 ? 0 : j;  // the sequence that this lane prepares and finishes
  const bool valid = b0 + own < p.B;
  float u = 0.f, dl = 0.f, gate = 1.f;
  if (valid) {
    const long long b = b0 + own;
    u = Elem<T>::to_f32(static_cast<const T*>(p.u)[b * p.u_ld + d]);
    dl = Elem<T>::to_f32(static_cast<const T*>(p.dt)[b * p.dt_ld + d]) + (p.dt_bias ? __ldg(p.dt_bias + d) : 0.f);
    if (p.z) gate = silu_f32(Elem<T>::to_f32(static_cast<const T*>(p.z)[b * p.z_ld + d]));
    if (p.softplus) dl = softplus_f32(dl);
  }
  const float du = dl * u;
  dl *= 2.f;  // kHalfLog2e's other half
  float2 A[NV][2];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p.A + (long long)d * p.N + 4 * (v * LPC + j)));
    A[v][0] = make_float2(a.x * kHalfLog2e, a.y * kHalfLog2e);
    A[v][1] = make_float2(a.z * kHalfLog2e, a.w * kHalfLog2e);
  }
  const T* bm_row = static_cast<const T*>(p.Bm) + b0 * p.bm_ld + g * p.N + 4 * j;
  const T* cm_row = static_cast<const T*>(p.Cm) + b0 * p.cm_ld + g * p.N + 4 * j;
  float4 bm[R][NV], cm[R][NV];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      bm[r][v] = cm[r][v] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (b0 + r < p.B) {
        bm[r][v] = load4(bm_row + r * p.bm_ld + 4 * LPC * v);
        cm[r][v] = load4(cm_row + r * p.cm_ld + 4 * LPC * v);
      }
    }
  float y[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const float rd = R == 1 ? dl : __shfl_sync(0xffffffffu, dl, r, LPC);
    const float ru = R == 1 ? du : __shfl_sync(0xffffffffu, du, r, LPC);
    const float2 rd2 = make_float2(rd, rd), ru2 = make_float2(ru, ru);
    float2 acc = make_float2(0.f, 0.f);
    if (b0 + r < p.B) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const float2 e0 = mul2(rd2, A[v][0]), e1 = mul2(rd2, A[v][1]);
        const float2 h0 = fma2(make_float2(exp2_approx(e0.x), exp2_approx(e0.y)), make_float2(h[r][v].x, h[r][v].y),
                               mul2(ru2, make_float2(bm[r][v].x, bm[r][v].y)));
        const float2 h1 = fma2(make_float2(exp2_approx(e1.x), exp2_approx(e1.y)), make_float2(h[r][v].z, h[r][v].w),
                               mul2(ru2, make_float2(bm[r][v].z, bm[r][v].w)));
        acc = fma2(h0, make_float2(cm[r][v].x, cm[r][v].y), acc);
        acc = fma2(h1, make_float2(cm[r][v].z, cm[r][v].w), acc);
        __stcs(reinterpret_cast<float4*>(state_out + r * state_row + 4 * LPC * v), make_float4(h0.x, h0.y, h1.x, h1.y));
      }
    }
    y[r] = acc.x + acc.y;
  }
  float sum;
  if constexpr (R == 1) {
    sum = y[0];
#pragma unroll
    for (int o = LPC / 2; o > 0; o /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  } else {
    sum = transposed_sum<LPC>(y, j);
  }
  if (valid && (R > 1 || j == 0)) {
    const float o = fmaf(p.skip ? __ldg(p.skip + d) : 0.f, u, sum) * gate;
    static_cast<T*>(p.out)[(b0 + own) * (long long)p.D + d] = Elem<T>::from_f32(o);
  }
}

// A prompt of a few tokens for many sequences and channels: the same lanes walk along it, the
// states in registers.  A tile of the scan's kernels would be mostly empty.  Bound by HBM for
// one token, by issue from a few on: 512 sequences of 1536 channels take 17 us and 15 us a token.
template <typename T, int LPC, int NV>
__global__ void __launch_bounds__(kStepThreads) ssm_walk_kernel(const SsmParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int j = threadIdx.x % LPC;
  const int d = blockIdx.x * (kStepThreads / LPC) + threadIdx.x / LPC, b = blockIdx.y;
  if (d >= p.D) return;  // whole warps: D is a multiple of 16
  const int len = p.lengths ? min(max(__ldg(p.lengths + b), 0), p.L) : p.L;
  const int g = d / (p.D / p.G);
  const float skip = p.skip ? __ldg(p.skip + d) : 0.f, bias = p.dt_bias ? __ldg(p.dt_bias + d) : 0.f;
  const long long state = ((long long)b * p.D + d) * p.N + 4 * j;
  float2 A[NV][2], h[NV][2];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p.A + (long long)d * p.N + 4 * (v * LPC + j)));
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (p.state_in) s = __ldcs(reinterpret_cast<const float4*>(p.state_in + state + 4 * LPC * v));
    A[v][0] = make_float2(a.x * kHalfLog2e, a.y * kHalfLog2e);
    A[v][1] = make_float2(a.z * kHalfLog2e, a.w * kHalfLog2e);
    h[v][0] = make_float2(s.x, s.y);
    h[v][1] = make_float2(s.z, s.w);
  }
  ScanWalk at(p.map, 0);
  for (int s = 0; s < len; ++s, at.next(p.map)) {
    const long long row = (long long)b * p.L + at.token;
    const float u = Elem<T>::to_f32(static_cast<const T*>(p.u)[row * p.u_ld + d]);
    float dl = Elem<T>::to_f32(static_cast<const T*>(p.dt)[row * p.dt_ld + d]) + bias;
    const float z = p.z ? Elem<T>::to_f32(static_cast<const T*>(p.z)[row * p.z_ld + d]) : 0.f;
    if (p.softplus) dl = softplus_f32(dl);
    const float du = dl * u;
    const float2 dl2 = make_float2(2.f * dl, 2.f * dl), du2 = make_float2(du, du);
    const T* bm_row = static_cast<const T*>(p.Bm) + row * p.bm_ld + g * p.N + 4 * j;
    const T* cm_row = static_cast<const T*>(p.Cm) + row * p.cm_ld + g * p.N + 4 * j;
    float2 acc = make_float2(0.f, 0.f);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const float4 bm = load4(bm_row + 4 * LPC * v), cm = load4(cm_row + 4 * LPC * v);
      const float2 e0 = mul2(dl2, A[v][0]), e1 = mul2(dl2, A[v][1]);
      h[v][0] = fma2(make_float2(exp2_approx(e0.x), exp2_approx(e0.y)), h[v][0], mul2(du2, make_float2(bm.x, bm.y)));
      h[v][1] = fma2(make_float2(exp2_approx(e1.x), exp2_approx(e1.y)), h[v][1], mul2(du2, make_float2(bm.z, bm.w)));
      acc = fma2(h[v][0], make_float2(cm.x, cm.y), acc);
      acc = fma2(h[v][1], make_float2(cm.z, cm.w), acc);
    }
    float y = acc.x + acc.y;
#pragma unroll
    for (int o = LPC / 2; o > 0; o /= 2) y += __shfl_xor_sync(0xffffffffu, y, o);
    y = fmaf(skip, u, y);
    if (p.z) y *= silu_f32(z);
    if (j == 0) static_cast<T*>(p.out)[row * p.D + d] = Elem<T>::from_f32(y);
  }
  if (p.state_out) {
#pragma unroll
    for (int v = 0; v < NV; ++v)
      __stcs(reinterpret_cast<float4*>(p.state_out + state + 4 * LPC * v),
             make_float4(h[v][0].x, h[v][0].y, h[v][1].x, h[v][1].y));
  }
}

template <typename T, int LPC, int NV>
gtr_status_t launch_step_v(const SsmParams& p, cudaStream_t stream) {
  constexpr int kCh = kStepThreads / LPC;
  const unsigned gx = (unsigned)((p.D + kCh - 1) / kCh);
  // LPC sequences a thread where they fill the GPU and the registers hold their states (bf16, LPC
  // and one, D = 1536: N = 16, 512 sequences 23.6 and 27.4 us, 64 4.3 and 4.8 us, 43 3.5 and 3.5
  // us; 4 sequences of D = 768 2.4 and 1.9 us; N = 64, 64 sequences 15.1 and 11.0 us)
  if constexpr (NV == 1) {
    if ((long long)p.B * p.D >= 64 * 1024)
      return launch_serial(ssm_step_kernel<T, LPC, NV, LPC>, dim3(gx, (unsigned)((p.B + LPC - 1) / LPC)),
                           dim3(kStepThreads), 0, stream, p);
  }
  return launch_serial(ssm_step_kernel<T, LPC, NV, 1>, dim3(gx, (unsigned)p.B), dim3(kStepThreads), 0, stream, p);
}

template <typename T, int LPC, int NV>
gtr_status_t launch_walk_v(const SsmParams& p, cudaStream_t stream) {
  constexpr int kCh = kStepThreads / LPC;
  return launch_serial(ssm_walk_kernel<T, LPC, NV>, dim3((unsigned)((p.D + kCh - 1) / kCh), (unsigned)p.B),
                       dim3(kStepThreads), 0, stream, p);
}

template <typename T>
gtr_status_t launch_step(const SsmParams& p, bool walk, cudaStream_t stream) {
#define GTR_BY_N(LPC, NV) (walk ? launch_walk_v<T, LPC, NV>(p, stream) : launch_step_v<T, LPC, NV>(p, stream))
  switch (p.N / 8) {  // four lanes where N is a multiple of 16
    case 1: return GTR_BY_N(2, 1);
    case 2: return GTR_BY_N(4, 1);
    case 3: return GTR_BY_N(2, 3);
    case 4: return GTR_BY_N(4, 2);
    case 5: return GTR_BY_N(2, 5);
    case 6: return GTR_BY_N(4, 3);
    case 7: return GTR_BY_N(2, 7);
    default: return GTR_BY_N(4, 4);
  }
#undef GTR_BY_N
}

gtr_status_t launch_typed(const SsmParams& p, int dtype, bool walk, cudaStream_t stream) {
  switch (dtype) {
    case GTR_F16: return launch_step<__half>(p, walk, stream);
    case GTR_BF16: return launch_step<__nv_bfloat16>(p, walk, stream);
    default: return launch_step<float>(p, walk, stream);
  }
}

}  // namespace

gtr_status_t launch_ssm_walk(const SsmParams& p, int dtype, cudaStream_t stream) {
  return launch_typed(p, dtype, true, stream);
}

gtr_status_t validate_ssm_shape(int B, int grid_H, int grid_W, int D, int N, int G, int dtype) {
  if (B <= 0 || grid_H <= 0 || grid_W <= 0 || D <= 0 || N <= 0 || G <= 0 || dtype < GTR_F32 || dtype > GTR_BF16 ||
      D % G != 0)
    return GTR_ERR_INVALID_ARG;
  const long long L = (long long)grid_H * grid_W;
  if (N % 8 != 0 || N > 64 || (D / G) % 16 != 0 || D > (1 << 20) || B > 65535 || L > (1ll << 28))
    return GTR_ERR_UNSUPPORTED;
  return GTR_OK;
}

gtr_status_t validate_ssm(const SsmParams& p, int grid_H, int grid_W, int direction, int dtype) {
  if (!p.u || !p.dt || !p.A || !p.Bm || !p.Cm || !p.out) return GTR_ERR_INVALID_ARG;
  if (direction < GTR_L2R || direction > GTR_B2T) return GTR_ERR_INVALID_ARG;
  const gtr_status_t shape = validate_ssm_shape(p.B, grid_H, grid_W, p.D, p.N, p.G, dtype);
  if (shape == GTR_ERR_INVALID_ARG) return shape;
  for (const void* q : {p.u, p.dt, p.Bm, p.Cm, p.z, (const void*)p.A, (const void*)p.state_in,
                        (const void*)p.state_out, (const void*)p.out})
    if (!aligned_to(q, 16)) return GTR_ERR_INVALID_ARG;
  if (!aligned_to(p.skip, 4) || !aligned_to(p.dt_bias, 4) || !aligned_to(p.lengths, 4)) return GTR_ERR_INVALID_ARG;
  const int es = dtype == GTR_F32 ? 4 : 2;
  const long long gn = (long long)p.G * p.N;
  if (p.u_ld < p.D || p.dt_ld < p.D || p.bm_ld < gn || p.cm_ld < gn || (p.z && p.z_ld < p.D)) return GTR_ERR_INVALID_ARG;
  for (long long ld : {p.u_ld, p.dt_ld, p.bm_ld, p.cm_ld, p.z ? p.z_ld : 0ll})
    if (ld % (16 / es) != 0) return GTR_ERR_INVALID_ARG;
  if (shape != GTR_OK) return shape;
  const long long rows = (long long)p.B * grid_H * grid_W;
  for (long long ld : {p.u_ld, p.dt_ld, p.bm_ld, p.cm_ld, p.z ? p.z_ld : 0ll})
    if (ld > (1ll << 32) || (double)rows * (double)ld >= 1e12) return GTR_ERR_UNSUPPORTED;
  const size_t no = span_bytes(rows, p.D, p.D, es), ns = (size_t)p.B * p.D * p.N * 4, na = (size_t)p.D * p.N * 4;
  const struct {
    const void* q;
    size_t n;
  } in[] = {{p.u, span_bytes(rows, p.u_ld, p.D, es)},    {p.dt, span_bytes(rows, p.dt_ld, p.D, es)},
            {p.Bm, span_bytes(rows, p.bm_ld, gn, es)},   {p.Cm, span_bytes(rows, p.cm_ld, gn, es)},
            {p.z, span_bytes(rows, p.z_ld, p.D, es)},    {p.A, na},
            {p.skip, (size_t)p.D * 4},                   {p.dt_bias, (size_t)p.D * 4},
            {p.lengths, (size_t)p.B * 4}};
  for (const auto& i : in)
    if (overlaps(p.out, no, i.q, i.n) || overlaps(p.state_out, ns, i.q, i.n)) return GTR_ERR_INVALID_ARG;
  if (overlaps(p.out, no, p.state_in, ns) || overlaps(p.out, no, p.state_out, ns) ||
      (p.state_in != p.state_out && overlaps(p.state_in, ns, p.state_out, ns)))
    return GTR_ERR_INVALID_ARG;
  return GTR_OK;
}

}  // namespace gtr

extern "C" gtr_status_t gtr_ssm_step(const void* u, int64_t u_ld, const void* dt, int64_t dt_ld, const float* A,
                                     const void* Bm, int64_t bm_ld, const void* Cm, int64_t cm_ld, const void* z,
                                     int64_t z_ld, const float* skip, const float* dt_bias, int softplus,
                                     const float* state_in, float* state_out, void* out, int B, int D, int N, int G,
                                     int dtype, gtr_stream_t stream) {
  using namespace gtr;
  if (!state_in || !state_out) return GTR_ERR_INVALID_ARG;
  const SsmParams p{u,     dt,    Bm,      Cm,       z,         u_ld,    dt_ld, bm_ld, cm_ld, z_ld, A,
                    skip,  dt_bias, state_in, state_out, nullptr, out,   B,     1,     D,     N,    G,
                    softplus != 0, ScanMap::make(GTR_L2R, 1, 1)};
  const gtr_status_t st = validate_ssm(p, 1, 1, GTR_L2R, dtype);
  if (st != GTR_OK) return st;
  return launch_typed(p, dtype, false, reinterpret_cast<cudaStream_t>(stream));
}
