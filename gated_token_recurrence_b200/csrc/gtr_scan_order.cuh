// The scan order as a walk: which token follows which, without a division per token.
#pragma once

#include "gtr.h"

namespace gtr {

// Position s = line * n + i of the scan is token line * line_stride + first + i * step (the
// four orders of scan_to_token).  A grid has at most 2^28 tokens, so int holds every value.
struct ScanMap {
  int n;            // positions per line
  int line_stride;  // tokens between lines
  int first, step;  // token of a line's first position; tokens between positions

  static __host__ __device__ ScanMap make(int dir, int H, int W) {
    switch (dir) {
      case GTR_L2R: return {W, W, 0, 1};
      case GTR_R2L: return {W, W, W - 1, -1};
      case GTR_T2B: return {H, 1, 0, W};
      default: return {H, 1, (H - 1) * W, -W};
    }
  }
  __host__ __device__ __forceinline__ int token(unsigned s) const {
    const unsigned line = s / (unsigned)n, i = s - line * (unsigned)n;
    return (int)line * line_stride + first + (int)i * step;
  }
};

// A walk along the scan from one position on.
struct ScanWalk {
  int i, token;
  __device__ __forceinline__ ScanWalk(const ScanMap& m, unsigned s) {
    const unsigned line = s / (unsigned)m.n;
    i = (int)(s - line * (unsigned)m.n);
    token = (int)line * m.line_stride + m.first + i * m.step;
  }
  __device__ __forceinline__ void next(const ScanMap& m) {
    token += m.step;
    if (++i == m.n) {
      i = 0;
      token += m.line_stride - m.n * m.step;
    }
  }
};

}  // namespace gtr
