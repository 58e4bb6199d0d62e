// Selective state space scan over a prompt, along one of the four scan directions.
#include "gtr_launch.cuh"
#include "gtr_ssm.cuh"
#include "gtr_ssm_host.h"

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
  return launch_ssm_chain(p, dtype, reinterpret_cast<cudaStream_t>(stream));
}
