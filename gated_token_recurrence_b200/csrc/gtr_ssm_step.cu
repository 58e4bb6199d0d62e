// Selective state space scan, one chain per channel: the form for single tokens.
//
// The recurrence of gtr_ssm.cuh with the N states of a channel spread over LPC neighbouring
// lanes, NV float4 each, so that a warp reads and writes the stored states in whole sectors;
// the output sum over n is a shuffle reduction of the LPC lanes.  For one token the traffic
// is the state, 8 N bytes per channel in and out, against 8 bytes (16-bit data) of u, dt, z
// and out: bound by HBM bandwidth.
#include "gtr_launch.cuh"
#include "gtr_ssm.cuh"
#include "gtr_ssm_host.h"

namespace gtr {
namespace {

constexpr int kStepThreads = 128;

template <typename T, int LPC, int NV>
__global__ void __launch_bounds__(kStepThreads) ssm_chain_kernel(const SsmParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int kCh = kStepThreads / LPC;
  const int j = threadIdx.x % LPC;
  const int d = blockIdx.x * kCh + threadIdx.x / LPC, b = blockIdx.y;
  if (d >= p.D) return;
  const unsigned mask = __activemask();  // the LPC lanes of a channel stay or leave together
  const int len = p.lengths ? min(max(__ldg(p.lengths + b), 0), p.L) : p.L;
  const float skip = p.skip ? __ldg(p.skip + d) : 0.f, bias = p.dt_bias ? __ldg(p.dt_bias + d) : 0.f;
  const int g = d / (p.D / p.G);
  float4 A[NV], h[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int n = 4 * (v * LPC + j);
    const float4 a = __ldg(reinterpret_cast<const float4*>(p.A + (long long)d * p.N + n));
    A[v] = make_float4(a.x * kLog2e, a.y * kLog2e, a.z * kLog2e, a.w * kLog2e);
    h[v] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (p.state_in) h[v] = *reinterpret_cast<const float4*>(p.state_in + ((long long)b * p.D + d) * p.N + n);
  }
  ScanWalk at(p.map, 0);
  for (int s = 0; s < len; ++s, at.next(p.map)) {
    const long long row = (long long)b * p.L + at.token;
    const float u = Elem<T>::to_f32(static_cast<const T*>(p.u)[row * p.u_ld + d]);
    float dl = Elem<T>::to_f32(static_cast<const T*>(p.dt)[row * p.dt_ld + d]) + bias;
    const float zg = p.z ? Elem<T>::to_f32(static_cast<const T*>(p.z)[row * p.z_ld + d]) : 0.f;
    if (p.softplus) dl = softplus_f32(dl);
    const float du = dl * u;
    float y = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int n = g * p.N + 4 * (v * LPC + j);
      const float4 bm = load4(static_cast<const T*>(p.Bm) + row * p.bm_ld + n);
      const float4 cm = load4(static_cast<const T*>(p.Cm) + row * p.cm_ld + n);
      h[v].x = fmaf(exp2_approx(dl * A[v].x), h[v].x, du * bm.x);
      h[v].y = fmaf(exp2_approx(dl * A[v].y), h[v].y, du * bm.y);
      h[v].z = fmaf(exp2_approx(dl * A[v].z), h[v].z, du * bm.z);
      h[v].w = fmaf(exp2_approx(dl * A[v].w), h[v].w, du * bm.w);
      y = fmaf(h[v].x, cm.x, fmaf(h[v].y, cm.y, fmaf(h[v].z, cm.z, fmaf(h[v].w, cm.w, y))));
    }
#pragma unroll
    for (int o = LPC / 2; o > 0; o >>= 1) y += __shfl_xor_sync(mask, y, o);
    y = fmaf(skip, u, y);
    if (p.z) y *= silu_f32(zg);
    if (j == 0) static_cast<T*>(p.out)[row * p.D + d] = Elem<T>::from_f32(y);
  }
  if (p.state_out) {
#pragma unroll
    for (int v = 0; v < NV; ++v)
      *reinterpret_cast<float4*>(p.state_out + ((long long)b * p.D + d) * p.N + 4 * (v * LPC + j)) = h[v];
  }
}

template <typename T, int LPC, int NV>
gtr_status_t launch_chain_v(const SsmParams& p, cudaStream_t stream) {
  constexpr int kCh = kStepThreads / LPC;
  return launch_serial(ssm_chain_kernel<T, LPC, NV>, dim3((unsigned)((p.D + kCh - 1) / kCh), (unsigned)p.B),
                       dim3(kStepThreads), 0, stream, p);
}

template <typename T>
gtr_status_t launch_chain_t(const SsmParams& p, cudaStream_t stream) {
  switch (p.N / 8) {
    case 1: return launch_chain_v<T, 2, 1>(p, stream);
    case 2: return launch_chain_v<T, 4, 1>(p, stream);
    case 3: return launch_chain_v<T, 2, 3>(p, stream);
    case 4: return launch_chain_v<T, 4, 2>(p, stream);
    case 5: return launch_chain_v<T, 2, 5>(p, stream);
    case 6: return launch_chain_v<T, 4, 3>(p, stream);
    case 7: return launch_chain_v<T, 2, 7>(p, stream);
    default: return launch_chain_v<T, 4, 4>(p, stream);
  }
}

}  // namespace

gtr_status_t launch_ssm_chain(const SsmParams& p, int dtype, cudaStream_t stream) {
  switch (dtype) {
    case GTR_F16: return launch_chain_t<__half>(p, stream);
    case GTR_BF16: return launch_chain_t<__nv_bfloat16>(p, stream);
    default: return launch_chain_t<float>(p, stream);
  }
}

gtr_status_t validate_ssm(const SsmParams& p, int grid_H, int grid_W, int direction, int dtype) {
  if (!p.u || !p.dt || !p.A || !p.Bm || !p.Cm || !p.out || p.B <= 0 || grid_H <= 0 || grid_W <= 0 || p.D <= 0 ||
      p.N <= 0 || p.G <= 0)
    return GTR_ERR_INVALID_ARG;
  if (direction < GTR_L2R || direction > GTR_B2T || dtype < GTR_F32 || dtype > GTR_BF16) return GTR_ERR_INVALID_ARG;
  for (const void* q : {p.u, p.dt, p.Bm, p.Cm, p.z, (const void*)p.A, (const void*)p.state_in,
                        (const void*)p.state_out, (const void*)p.out})
    if (!aligned_to(q, 16)) return GTR_ERR_INVALID_ARG;
  if (!aligned_to(p.skip, 4) || !aligned_to(p.dt_bias, 4) || !aligned_to(p.lengths, 4)) return GTR_ERR_INVALID_ARG;
  const int es = dtype == GTR_F32 ? 4 : 2;
  const long long gn = (long long)p.G * p.N;
  if (p.u_ld < p.D || p.dt_ld < p.D || p.bm_ld < gn || p.cm_ld < gn || (p.z && p.z_ld < p.D)) return GTR_ERR_INVALID_ARG;
  for (long long ld : {p.u_ld, p.dt_ld, p.bm_ld, p.cm_ld, p.z ? p.z_ld : 0ll})
    if (ld % (16 / es) != 0) return GTR_ERR_INVALID_ARG;
  if (p.D % p.G != 0) return GTR_ERR_INVALID_ARG;
  const long long L = (long long)grid_H * grid_W;
  if (p.N % 8 != 0 || p.N > 64 || (p.D / p.G) % 16 != 0 || p.D > (1 << 20) || p.B > 65535 || L > (1ll << 28))
    return GTR_ERR_UNSUPPORTED;
  const long long rows = p.B * L;
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
  return launch_ssm_chain(p, dtype, reinterpret_cast<cudaStream_t>(stream));
}
