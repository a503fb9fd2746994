// router_math.cuh -- what every kernel that reads the router's state shares:
// the affinities from the logit partials, and a token's packed sequence.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

constexpr int EPL = 8;  // experts per lane (N_r <= 256)

// s_{e,t} from the router's logit partials: the K splits are added in split
// order, then the sigmoid.  Every kernel that needs the affinities computes
// them here, so they agree bit for bit.
__device__ __forceinline__ float affinity(const float *__restrict__ partial, int n_ks, int64_t T, int Nr,
                                          int64_t t, int e) {
  float z = 0.0f;
  for (int k = 0; k < n_ks; ++k) z += partial[(static_cast<int64_t>(k) * T + t) * Nr + e];
  return 1.0f / (1.0f + expf(-z));
}

// s and 1 - s.  For z >= 0, 1 - s = e^-z s (1 - s itself would cancel); below,
// s < 1/2 and the difference keeps its digits.
__device__ __forceinline__ void affinity_pair(const float *__restrict__ partial, int n_ks, int64_t T, int Nr,
                                              int64_t t, int e, float &s, float &om) {
  float z = 0.0f;
  for (int k = 0; k < n_ks; ++k) z += partial[(static_cast<int64_t>(k) * T + t) * Nr + e];
  const float q = expf(-z);
  s = 1.0f / (1.0f + q);
  om = z >= 0.0f ? q * s : 1.0f - s;
}

// The first sequence that ends behind token t (n_seq if none does): sequence
// s holds the tokens [off[s], off[s + 1]).  Offsets come from device memory
// and may be wrong: whatever they hold, the result is in [0, n_seq].
__device__ __forceinline__ int seq_of(const int32_t *__restrict__ off, int n_seq, int64_t t) {
  int lo = 0, hi = n_seq;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (off[mid + 1] > t)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

}  // namespace moe
