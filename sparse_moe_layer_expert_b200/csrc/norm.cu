// norm.cu -- what feeds the layer and takes its gradient back: residual
// addition + RMS norm + 1x128 FP8 quantization in one pass, and its backward.
//
// Forward, per row (token) of `cols` channels:
//   h = x + resid, rounded to the residual stream's type (bf16 or FP32);
//   rstd = 1 / sqrt(mean(h^2) + eps);  y = h rstd w            (FP32)
//   y is stored as bf16 (the router's input); each 128-channel tile of the
//   FP32 y -- not of its bf16 copy, which would round twice -- is quantized
//   as in quant.cu (S = amax / 448 or a power of two, E4M3 codes of y / S).
// A row stays in registers from the one read of x and resid to the writes of
// h, y and the codes; the sum of squares and the tile maxima are FP32.
//
// Backward, with n = h rstd and g = dy w:
//   dx = dres + rstd (g - n mean(g n))   (the gradient of x and of resid alike)
//   dw = sum over rows of dy n
// dw is summed per CTA in registers over the CTA's rows, then over the CTAs in
// CTA order by a second kernel: no atomics, the same result on every run.
#include "common.cuh"
#include "kernels.h"

namespace moe {

namespace {

// ---------------------------------------------------------- 8-value chunks
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&f)[8]) {
  const uint4 v = *reinterpret_cast<const uint4 *>(p);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void load8(const float *p, float (&f)[8]) {
  const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
  f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}
__device__ __forceinline__ uint4 pack_bf16x8(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b2 = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&b2);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&f)[8]) {
  *reinterpret_cast<uint4 *>(p) = pack_bf16x8(f);
}
__device__ __forceinline__ void store8(float *p, const float (&f)[8]) {
  reinterpret_cast<float4 *>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4 *>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}
// h rounded to the stream's type (the value later readers of h see)
__device__ __forceinline__ void round8(const __nv_bfloat16 *, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = __bfloat162float(__float2bfloat16_rn(f[i]));
}
__device__ __forceinline__ void round8(const float *, float (&)[8]) {}

// Sum over the threads of one row (threadIdx.x; blockDim.x a multiple of 32):
// a butterfly in each warp, then the warps' sums in warp order.  Every thread
// of the block calls it; buf holds blockDim.y x 32 floats.  A row's result is
// the same in all its threads.
__device__ __forceinline__ float row_sum(float v, float *buf) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int nw = blockDim.x >> 5;
  if (nw == 1) return v;
  if ((threadIdx.x & 31) == 0) buf[threadIdx.y * 32 + (threadIdx.x >> 5)] = v;
  __syncthreads();
  float s = 0.0f;
  for (int i = 0; i < nw; ++i) s += buf[threadIdx.y * 32 + i];
  return s;
}

// Codes of 8 values of a tile with scale S (see codes8 in quant.cu); a
// non-finite S gives NaN codes.
__device__ __forceinline__ uint2 tile_codes(const float (&f)[8], float S) {
  uint32_t lo = 0, hi = 0;
  if (S >= 0x1p-100f) {
    const float r = __frcp_rn(S);
    lo = e4m3x2_rn_sat(div_by_recip(f[0], S, r), div_by_recip(f[1], S, r)) |
         (e4m3x2_rn_sat(div_by_recip(f[2], S, r), div_by_recip(f[3], S, r)) << 16);
    hi = e4m3x2_rn_sat(div_by_recip(f[4], S, r), div_by_recip(f[5], S, r)) |
         (e4m3x2_rn_sat(div_by_recip(f[6], S, r), div_by_recip(f[7], S, r)) << 16);
  } else if (S != 0.0f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) lo |= static_cast<uint32_t>(e4m3_rn_sat(f[i] / S)) << (8 * i);
#pragma unroll
    for (int i = 0; i < 4; ++i) hi |= static_cast<uint32_t>(e4m3_rn_sat(f[4 + i] / S)) << (8 * i);
  }
  return make_uint2(lo, hi);
}

struct NormFwd {
  const void *x, *resid;
  int64_t ld_x, ld_r;
  const float *w;
  float eps;
  int64_t rows;
  int cols;
  void *h;
  __nv_bfloat16 *y;
  uint8_t *q;
  float *s;
  float *rstd;
};

}  // namespace

// blockDim = (threads per row, rows per CTA); thread tx of a row holds the
// 8-channel chunks tx, tx + blockDim.x, ... (CH of them at most), so every
// 16 lanes hold one 128-channel tile.
template <typename TS, int CH, bool POW2, int MAXT>
__global__ void __launch_bounds__(MAXT, 1) add_rmsnorm_quant_kernel(const NormFwd p) {
  __shared__ float buf[8 * 32];
  const int64_t r = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  const bool live = r < p.rows;
  const int nch = p.cols / 8;
  float f[CH][8];
  float ss = 0.0f;
  const TS *x = static_cast<const TS *>(p.x) + r * p.ld_x;
  const TS *rs = p.resid ? static_cast<const TS *>(p.resid) + r * p.ld_r : nullptr;
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int c = threadIdx.x + k * blockDim.x;
#pragma unroll
    for (int i = 0; i < 8; ++i) f[k][i] = 0.0f;
    if (live && c < nch) {
      load8(x + c * 8, f[k]);
      if (rs) {
        float g[8];
        load8(rs + c * 8, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[k][i] += g[i];
        round8(x, f[k]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(f[k][i], f[k][i], ss);
    }
  }
  ss = row_sum(ss, buf);
  const float rstd = 1.0f / sqrtf(ss / static_cast<float>(p.cols) + p.eps);
  if (live && threadIdx.x == 0 && p.rstd) p.rstd[r] = rstd;
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int c = threadIdx.x + k * blockDim.x;
    // a tile's 16 lanes are all inside or all outside the row
    const bool in = live && c < nch;
    if (in && p.h) store8(static_cast<TS *>(p.h) + r * p.cols + c * 8, f[k]);
    uint32_t am = 0;
    if (in) {
      float w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = 1.0f;
      if (p.w) load8(p.w + c * 8, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        f[k][i] = f[k][i] * rstd * w[i];
        // as integers, |NaN| > |inf| > every finite magnitude
        am = max(am, __float_as_uint(f[k][i]) & 0x7FFFFFFFu);
      }
      if (p.y) store8(p.y + r * p.cols + c * 8, f[k]);
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) am = max(am, __shfl_xor_sync(0xffffffffu, am, o));
    const float amax = __uint_as_float(am);
    float S = POW2 ? pow2_scale(amax) : amax / 448.0f;
    if (am >= 0x7F800000u) S = __uint_as_float(0x7FFFFFFFu);
    if (in) {
      *reinterpret_cast<uint2 *>(p.q + r * p.cols + c * 8) = tile_codes(f[k], S);
      if ((threadIdx.x & 15) == 0) p.s[r * (p.cols / 128) + (c >> 4)] = S;
    }
  }
}

namespace {
struct NormBwd {
  const void *dy, *h, *dres;
  const float *w, *rstd;
  int64_t rows;
  int cols;
  void *dx;
  float *dw_part;  // [gridDim.x, cols]
};
}  // namespace

template <typename TY, typename TS, typename TX, int CH, int MAXT>
__global__ void __launch_bounds__(MAXT, 1) add_rmsnorm_bwd_kernel(const NormBwd p) {
  __shared__ float buf[2][8 * 32];
  extern __shared__ float dw_sh[];  // [blockDim.y, cols] when a CTA holds several rows
  const int nch = p.cols / 8;
  float dw[CH][8];
#pragma unroll
  for (int k = 0; k < CH; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[k][i] = 0.0f;
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.y;
  int ph = 0;
  // every thread of the CTA makes the same number of turns (row_sum is a CTA barrier)
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * blockDim.y; r0 < p.rows; r0 += step, ph ^= 1) {
    const int64_t r = r0 + threadIdx.y;
    const bool live = r < p.rows;
    float n[CH][8], g[CH][8];
    float sum = 0.0f;
    const float rstd = live ? p.rstd[r] : 0.0f;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = threadIdx.x + k * blockDim.x;
      if (live && c < nch) {
        load8(static_cast<const TS *>(p.h) + r * p.cols + c * 8, n[k]);
        load8(static_cast<const TY *>(p.dy) + r * p.cols + c * 8, g[k]);
        float w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = 1.0f;
        if (p.w) load8(p.w + c * 8, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          n[k][i] *= rstd;
          dw[k][i] = fmaf(g[k][i], n[k][i], dw[k][i]);
          g[k][i] *= w[i];
          sum = fmaf(g[k][i], n[k][i], sum);
        }
      }
    }
    // two buffers in turn: a row's sums are read while the next row's are written
    const float m = row_sum(sum, buf[ph]) / static_cast<float>(p.cols);
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = threadIdx.x + k * blockDim.x;
      if (live && c < nch) {
        float d[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = 0.0f;
        if (p.dres) load8(static_cast<const TS *>(p.dres) + r * p.cols + c * 8, d);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = fmaf(rstd, fmaf(-n[k][i], m, g[k][i]), d[i]);
        store8(static_cast<TX *>(p.dx) + r * p.cols + c * 8, d);
      }
    }
  }
  if (!p.dw_part) return;
  float *part = p.dw_part + static_cast<int64_t>(blockIdx.x) * p.cols;
  if (blockDim.y == 1) {
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = threadIdx.x + k * blockDim.x;
      if (c < nch) store8(part + c * 8, dw[k]);
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int c = threadIdx.x + k * blockDim.x;
    if (c < nch) store8(dw_sh + threadIdx.y * p.cols + c * 8, dw[k]);
  }
  __syncthreads();
  for (int c = threadIdx.y * blockDim.x + threadIdx.x; c < p.cols; c += blockDim.x * blockDim.y) {
    float s = 0.0f;
    for (int y = 0; y < static_cast<int>(blockDim.y); ++y) s += dw_sh[y * p.cols + c];
    part[c] = s;
  }
}

// dw[c] = sum over the parts, 32 columns per CTA: each of 32 warps takes every
// 32nd part, then the warps' sums are added in warp order.
__global__ void __launch_bounds__(1024) norm_dw_join_kernel(const float *__restrict__ part, int n_part, int cols,
                                                             float *__restrict__ dw) {
  __shared__ float sh[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.0f;
  for (int i = warp; i < n_part; i += 32) s += part[static_cast<int64_t>(i) * cols + c];
  sh[warp][lane] = s;
  __syncthreads();
  if (warp == 0) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) t += sh[i][lane];
    dw[c] = t;
  }
}

namespace {
// Threads per row for CH chunks each, and rows per CTA (about 256 threads).
inline dim3 norm_block(int cols, int ch) {
  const int nch = cols / 8;
  const int tx = ((nch + ch - 1) / ch + 31) / 32 * 32;
  int ty = 256 / tx;
  if (ty < 1) ty = 1;
  if (ty > 8) ty = 8;
  return dim3(static_cast<unsigned>(tx), static_cast<unsigned>(ty));
}

// Rows of up to 8192 channels take at most 256 threads, which leaves the
// registers for CH = 4 chunks a thread; longer rows take up to 1024.
constexpr int kCh = 4;

template <typename TS, bool POW2>
cudaError_t launch_norm_fwd(const NormFwd &p, cudaStream_t st) {
  const dim3 b = norm_block(p.cols, kCh);
  const unsigned grid = static_cast<unsigned>((p.rows + b.y - 1) / b.y);
  if (b.x <= 256)
    add_rmsnorm_quant_kernel<TS, kCh, POW2, 256><<<grid, b, 0, st>>>(p);
  else
    add_rmsnorm_quant_kernel<TS, kCh, POW2, 1024><<<grid, b, 0, st>>>(p);
  return cudaGetLastError();
}

template <typename TY, typename TS, typename TX>
cudaError_t launch_norm_bwd(const NormBwd &p, int grid, cudaStream_t st) {
  const dim3 b = norm_block(p.cols, kCh);
  const size_t sh = b.y > 1 ? static_cast<size_t>(b.y) * p.cols * 4 : 0;  // 32 KB at most
  if (b.x <= 256)
    add_rmsnorm_bwd_kernel<TY, TS, TX, kCh, 256><<<grid, b, sh, st>>>(p);
  else
    add_rmsnorm_bwd_kernel<TY, TS, TX, kCh, 1024><<<grid, b, sh, st>>>(p);
  return cudaGetLastError();
}
}  // namespace

cudaError_t launch_add_rmsnorm_quant(const void *x, int64_t ld_x, const void *resid, int64_t ld_r, bool f32,
                                     const float *w, float eps, int64_t rows, int cols, void *h, void *y, uint8_t *q,
                                     float *s, float *rstd, bool pow2, cudaStream_t st) {
  if (rows == 0) return cudaSuccess;
  NormFwd p{x, resid, ld_x, ld_r, w, eps, rows, cols, h, static_cast<__nv_bfloat16 *>(y), q, s, rstd};
  using B = __nv_bfloat16;
  return f32 ? (pow2 ? launch_norm_fwd<float, true>(p, st) : launch_norm_fwd<float, false>(p, st))
             : (pow2 ? launch_norm_fwd<B, true>(p, st) : launch_norm_fwd<B, false>(p, st));
}

int norm_bwd_parts(int64_t rows, int cols) {
  const dim3 b = norm_block(cols, kCh);
  const int64_t want = (rows + b.y - 1) / b.y;
  const int64_t most = 2 * static_cast<int64_t>(moe_host::sm_count());
  return static_cast<int>(want < most ? want : most);
}

cudaError_t launch_add_rmsnorm_bwd(const void *dy, bool dy_f32, const void *h, const void *dres, bool f32,
                                   const float *w, const float *rstd, int64_t rows, int cols, void *dx, bool dx_f32,
                                   float *dw, float *part, cudaStream_t st) {
  if (rows == 0) return dw ? cudaMemsetAsync(dw, 0, sizeof(float) * cols, st) : cudaSuccess;
  const NormBwd p{dy, h, dres, w, rstd, rows, cols, dx, dw ? part : nullptr};
  const int grid = norm_bwd_parts(rows, cols);
  using B = __nv_bfloat16;
  cudaError_t e;
  if (dy_f32)
    e = f32 ? (dx_f32 ? launch_norm_bwd<float, float, float>(p, grid, st) : launch_norm_bwd<float, float, B>(p, grid, st))
            : (dx_f32 ? launch_norm_bwd<float, B, float>(p, grid, st) : launch_norm_bwd<float, B, B>(p, grid, st));
  else
    e = f32 ? (dx_f32 ? launch_norm_bwd<B, float, float>(p, grid, st) : launch_norm_bwd<B, float, B>(p, grid, st))
            : (dx_f32 ? launch_norm_bwd<B, B, float>(p, grid, st) : launch_norm_bwd<B, B, B>(p, grid, st));
  if (e != cudaSuccess || !dw) return e;
  norm_dw_join_kernel<<<cols / 32, 1024, 0, st>>>(part, grid, cols, dw);
  return cudaGetLastError();
}

}  // namespace moe
