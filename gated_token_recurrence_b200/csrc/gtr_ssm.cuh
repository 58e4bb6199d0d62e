// What the selective scan's kernels share: the problem and the per-token scalar functions.
#pragma once

#include "gtr_common.cuh"
#include "gtr_math.cuh"
#include "gtr_scan_order.cuh"

namespace gtr {

// Per (sequence b, channel d), with s the position in the scan order and N states:
//     delta_s  = softplus(dt_s + dt_bias_d)                    (or dt_s + dt_bias_d)
//     h_s[n]   = exp(delta_s A_d[n]) h_{s-1}[n] + delta_s u_s B_s[n]
//     out_s    = ( sum_n C_s[n] h_s[n] + skip_d u_s ) SiLU(z_s)
struct SsmParams {
  const void* u;
  const void* dt;
  const void* Bm;  // rows [G][N]
  const void* Cm;
  const void* z;  // or nullptr
  long long u_ld, dt_ld, bm_ld, cm_ld, z_ld;  // elements between tokens
  const float* A;         // [D][N]
  const float* skip;      // [D] or nullptr
  const float* dt_bias;   // [D] or nullptr
  const float* state_in;  // [B][D][N] or nullptr
  float* state_out;       // [B][D][N] or nullptr; may be state_in
  const int* lengths;     // [B] or nullptr
  void* out;              // [B][L][D]
  int B, L, D, N, G, softplus;
  ScanMap map;
};

// log(1 + exp(x)) = max(x, 0) + log1p(e) with e = exp(-|x|) in (0, 1].  Steps are small (a
// thousandth is common), so the relative error matters: the exponential carries the rounding
// of its argument as a first-order correction, and log1p(e) = e q(e) with q of degree 9 fitted to
// log1p(e) / e on [0, 1] by least squares reweighted towards the largest relative error (Lawson's
// iteration): 5e-9 off, 1.5e-7 with its coefficients and Horner steps in fp32.
__device__ __forceinline__ float softplus_f32(float x) {
  const float a = fmaxf(-fabsf(x), -100.f);  // e^-100 is 0 in fp32; an infinite x stays out of the products
  const float hi = a * kLog2e;
  const float lo = fmaf(a, kLog2e, -hi) + a * 1.925963033500e-8f;  // log2(e) = kLog2e + 1.9259...e-8
  const float e0 = exp2_approx(hi);
  const float e = fmaf(e0, lo * 0.69314718f, e0);
  float q = -0.0032440212f;
  q = fmaf(q, e, 0.019851444f);
  q = fmaf(q, e, -0.0569594987f);
  q = fmaf(q, e, 0.106036514f);
  q = fmaf(q, e, -0.153055906f);
  q = fmaf(q, e, 0.196759388f);
  q = fmaf(q, e, -0.249541342f);
  q = fmaf(q, e, 0.333299637f);
  q = fmaf(q, e, -0.499999017f);
  q = fmaf(q, e, 1.f);
  return fmaf(e, q, x < 0.f ? 0.f : x);  // a NaN stays one
}

}  // namespace gtr
