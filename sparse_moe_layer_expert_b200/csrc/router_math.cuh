// router_math.cuh -- what every kernel that reads the router's state shares:
// the affinities from the logit partials, and a token's packed sequence.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

constexpr int EPL = 8;  // experts per lane (N_r <= 256)

// s_{e,t} from the router's logit partials: the K splits are added in split
// order, then the sigmoid; what selects and gates, and what moe_seq_balance_loss
// adds up, takes them from here.  (sigmoid_pair() is within a step of it.)
__device__ __forceinline__ float affinity(const float *__restrict__ partial, int n_ks, int64_t T, int Nr,
                                          int64_t t, int e) {
  float z = 0.0f;
  for (int k = 0; k < n_ks; ++k) z += partial[(static_cast<int64_t>(k) * T + t) * Nr + e];
  return 1.0f / (1.0f + expf(-z));
}

// A warp's view of one token's N_r <= 256 experts: lane l holds the experts
// 128 g + 4 l + j as element 4 g + j (g = 0, 1; j = 0..3), so a row is read
// and written 16 bytes a lane.
__device__ __forceinline__ int lane_expert(int lane, int i) { return (i >> 2) * 128 + lane * 4 + (i & 3); }

// The token's logits: the K splits are added in split order (as affinity()),
// B splits' loads under way at once at least.  VEC: N_r % 4 == 0 (16-byte loads).
// Experts behind N_r give 0.  B = 1 where the router has few splits, as it does
// for many tokens; with B = 4 a kernel takes twice the registers, which only
// pays where few tokens (and 4 to 16 splits) leave the SMs' registers free.
template <bool VEC, int B>
__device__ __forceinline__ void add_splits(const float *__restrict__ row, int64_t pitch, int Nr, int lane,
                                           float (&z)[EPL]) {
  if (VEC) {
    float4 v[B][2];
#pragma unroll
    for (int k = 0; k < B; ++k)
#pragma unroll
      for (int g = 0; g < 2; ++g)
        if (g * 128 + lane * 4 < Nr)
          v[k][g] = __ldg(reinterpret_cast<const float4 *>(row + k * pitch + g * 128 + lane * 4));
#pragma unroll
    for (int k = 0; k < B; ++k)
#pragma unroll
      for (int g = 0; g < 2; ++g)
        if (g * 128 + lane * 4 < Nr) {
          z[4 * g] += v[k][g].x;
          z[4 * g + 1] += v[k][g].y;
          z[4 * g + 2] += v[k][g].z;
          z[4 * g + 3] += v[k][g].w;
        }
  } else {
    float v[B][EPL];
#pragma unroll
    for (int k = 0; k < B; ++k)
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (lane_expert(lane, i) < Nr) v[k][i] = __ldg(row + k * pitch + lane_expert(lane, i));
#pragma unroll
    for (int k = 0; k < B; ++k)
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (lane_expert(lane, i) < Nr) z[i] += v[k][i];
  }
}

template <bool VEC, int B>
__device__ __forceinline__ void load_logits(const float *__restrict__ partial, int n_ks, int64_t T, int Nr, int64_t t,
                                            int lane, float (&z)[EPL]) {
#pragma unroll
  for (int i = 0; i < EPL; ++i) z[i] = 0.0f;
  const int64_t pitch = T * Nr;
  const float *row = partial + t * Nr;
  int k = 0;
  if (B > 1)
    for (; k + B <= n_ks; k += B) add_splits<VEC, B>(row + k * pitch, pitch, Nr, lane, z);
#pragma unroll 2
  for (; k < n_ks; ++k) add_splits<VEC, 1>(row + k * pitch, pitch, Nr, lane, z);
}

// One expert's logit, in the same order.
template <int B>
__device__ __forceinline__ float load_logit(const float *__restrict__ partial, int n_ks, int64_t T, int Nr, int64_t t,
                                            int e) {
  const int64_t pitch = T * Nr;
  const float *p = partial + t * Nr + e;
  float z = 0.0f;
  int k = 0;
  if (B > 1)
    for (; k + B <= n_ks; k += B) {
      float v[B];
#pragma unroll
      for (int i = 0; i < B; ++i) v[i] = __ldg(p + (k + i) * pitch);
#pragma unroll
      for (int i = 0; i < B; ++i) z += v[i];
    }
  for (; k < n_ks; ++k) z += __ldg(p + k * pitch);
  return z;
}

// s and 1 - s.  For z >= 0, 1 - s = e^-z s (1 - s itself would cancel); below,
// s < 1/2 and the difference keeps its digits.  The reciprocal is the hardware's,
// one FP32 step off at most where affinity()'s is half of one: it feeds gradients
// and sums of shares, not the selection (the IEEE one: 30.9 us a loss with its
// gradient at 16384 x 256, this one 27.2).  1 + q is taken 2^-24 times, so that
// the subnormal s of -88.7 < z < -87.3 is not flushed.
__device__ __forceinline__ void sigmoid_pair(float z, float &s, float &om) {
  const float q = expf(-z);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(fmaf(q, 0x1p-24f, 0x1p-24f)));  // q = inf gives 0
  s *= 0x1p-24f;
  om = z >= 0.0f ? q * s : 1.0f - s;
}

// 1 / sum of a token's affinities (0 if all of them are 0: every logit far below
// the exponential's range, and no share); finite for the smallest sum too, 2^-128.
__device__ __forceinline__ float share_scale(float sum) {
  return sum > 0.0f ? fminf(1.0f / sum, 3.402823466e38f) : 0.0f;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The first sequence that ends behind token t (n_seq if none does): sequence
// s holds the tokens [off[s], off[s + 1]).  A warp searches together, 32 probes
// a step.  Offsets come from device memory and may be wrong: whatever they
// hold, the result is in [0, n_seq], and its end is behind t if it is below
// n_seq.
__device__ __forceinline__ int seq_of(const int32_t *__restrict__ off, int n_seq, int64_t t, int lane) {
  int lo = 0, n = n_seq;  // the answer is in [lo, lo + n]
  while (n > 0) {
    const int step = (n + 31) / 32;
    const int last = (lane + 1) * step - 1;  // of this lane's group of sequences
    const bool before = last < n && off[lo + last + 1] <= t;
    const uint32_t not_before = ~__ballot_sync(0xffffffffu, before);
    const int c = not_before ? __ffs(not_before) - 1 : 32;  // groups that end at or before t
    const bool whole = (c + 1) * step <= n;                  // group c's last sequence was probed: it ends behind t
    lo += c * step;
    n = whole ? step - 1 : n - c * step;
  }
  return lo;
}

}  // namespace moe
