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
#include "operators.cuh"

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
  if ((reinterpret_cast<uintptr_t>(p) & 31) == 0) {
    st_f32x8(p, f);
  } else {  // a tensor that starts 16 bytes into a sector
    reinterpret_cast<float4 *>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
}
// The same from shared memory.  FP32: lanes 4..7 of every eight take their
// upper 16 bytes first, so that eight lanes 32 bytes apart meet all the banks.
__device__ __forceinline__ void load8_sh(const __nv_bfloat16 *p, float (&f)[8]) { load8(p, f); }
__device__ __forceinline__ void load8_sh(const float *p, float (&f)[8]) {
  const bool up = (threadIdx.x >> 2) & 1;
  const float4 a = reinterpret_cast<const float4 *>(p)[up ? 1 : 0], b = reinterpret_cast<const float4 *>(p)[up ? 0 : 1];
  f[0] = up ? b.x : a.x, f[1] = up ? b.y : a.y, f[2] = up ? b.z : a.z, f[3] = up ? b.w : a.w;
  f[4] = up ? a.x : b.x, f[5] = up ? a.y : b.y, f[6] = up ? a.z : b.z, f[7] = up ? a.w : b.w;
}
// Two FP32 operations an instruction, each rounded to nearest.
__device__ __forceinline__ void mul2(float &a0, float &a1, float b0, float b1) {
  uint64_t a, b;
  asm("mov.b64 %0, {%1, %2};" : "=l"(a) : "f"(a0), "f"(a1));
  asm("mov.b64 %0, {%1, %2};" : "=l"(b) : "f"(b0), "f"(b1));
  asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(a) : "l"(b));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a0), "=f"(a1) : "l"(a));
}
__device__ __forceinline__ void mul8(float (&a)[8], const float (&b)[8]) {
#pragma unroll
  for (int i = 0; i < 8; i += 2) mul2(a[i], a[i + 1], b[i], b[i + 1]);
}
__device__ __forceinline__ void mul8(float (&a)[8], float b) {
#pragma unroll
  for (int i = 0; i < 8; i += 2) mul2(a[i], a[i + 1], b, b);
}

// One chunk of h = x + resid, rounded to the stream's type, in FP32; and the
// chunk as it is stored.  In bf16 the packed addition rounds the exact sum once;
// adding in FP32 first changes nothing (a sum of two bf16 values that FP32
// cannot hold is further from a bf16 tie than FP32's rounding).
struct BfChunk {
  uint4 v;
};
struct F32Chunk {
  float4 a, b;
};
__device__ __forceinline__ void stream_sum(const __nv_bfloat16 *x, const __nv_bfloat16 *r, float (&f)[8], BfChunk &c) {
  c.v = *reinterpret_cast<const uint4 *>(x);
  uint32_t w[4] = {c.v.x, c.v.y, c.v.z, c.v.w};
  if (r) {
    const uint4 g = *reinterpret_cast<const uint4 *>(r);
    const uint32_t u[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 t = __hadd2_rn(*reinterpret_cast<const __nv_bfloat162 *>(&w[i]),
                                          *reinterpret_cast<const __nv_bfloat162 *>(&u[i]));
      w[i] = *reinterpret_cast<const uint32_t *>(&t);
    }
    c.v = make_uint4(w[0], w[1], w[2], w[3]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
template <bool SHARED>
__device__ __forceinline__ void stream_sum_f32(const float *x, const float *r, float (&f)[8]) {
  if (SHARED)
    load8_sh(x, f);
  else
    load8(x, f);
  if (r) {
    float g[8];
    if (SHARED)
      load8_sh(r, g);
    else
      load8(r, g);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] += g[i];
  }
}
__device__ __forceinline__ void store_h(__nv_bfloat16 *p, const float (&)[8], const BfChunk &c) {
  *reinterpret_cast<uint4 *>(p) = c.v;
}
__device__ __forceinline__ void store_h(float *p, const float (&f)[8], const F32Chunk &) { store8(p, f); }
template <bool SHARED>
__device__ __forceinline__ void load_h(const __nv_bfloat16 *x, const __nv_bfloat16 *r, float (&f)[8], BfChunk &c) {
  stream_sum(x, r, f, c);
}
template <bool SHARED>
__device__ __forceinline__ void load_h(const float *x, const float *r, float (&f)[8], F32Chunk &) {
  stream_sum_f32<SHARED>(x, r, f);
}
template <typename TS>
struct ChunkOf {
  using type = F32Chunk;
};
template <>
struct ChunkOf<__nv_bfloat16> {
  using type = BfChunk;
};

__device__ __forceinline__ float sum_sq(const float (&f)[8], float ss) {
  float o = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; i += 2) ffma2_vec(ss, o, f[i], f[i + 1], f[i], f[i + 1]);
  return ss + o;
}

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

// a <- -(a / S), the IEEE quotient as div_by_recip forms it, two values an
// instruction; ny = -RN(1 / S).  With the quotient negated throughout, the
// residual step keeps the sign of a zero without a copysign: a = -0 gives
// residual +0 and (+0) ny + (+0) = +0, the negative of -0.
__device__ __forceinline__ void neg_quot2(float &a0, float &a1, float S, float ny) {
  uint64_t a, q, r, s2, n2;
  asm("mov.b64 %0, {%1, %2};" : "=l"(a) : "f"(a0), "f"(a1));
  asm("mov.b64 %0, {%1, %1};" : "=l"(s2) : "f"(S));
  asm("mov.b64 %0, {%1, %1};" : "=l"(n2) : "f"(ny));
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(q) : "l"(a), "l"(n2));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(s2), "l"(q), "l"(a));  // what the quotient leaves of a
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(q) : "l"(r), "l"(n2), "l"(q));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a0), "=f"(a1) : "l"(q));
}

// Codes of 8 values of a tile with scale S: those of the correctly rounded
// quotients y / S, as in quant.cu.  A power of two scales exactly, so one
// product serves there; a tiny S, whose reciprocal overflows, takes the
// division, and a NaN one gives NaN codes.  (y times the reciprocal alone moved
// one code in a few million by a step; the two operations more are hidden
// behind the memory traffic.)
template <bool POW2>
__device__ __forceinline__ uint2 tile_codes(float (&f)[8], float S) {
  uint32_t lo = 0, hi = 0;
  if (S >= 0x1p-100f) {
    const float r = __frcp_rn(S);
    if (POW2) {
      mul8(f, r);
    } else {
#pragma unroll
      for (int i = 0; i < 8; i += 2) neg_quot2(f[i], f[i + 1], S, -r);
    }
    lo = e4m3x2_rn_sat(f[0], f[1]) | (e4m3x2_rn_sat(f[2], f[3]) << 16);
    hi = e4m3x2_rn_sat(f[4], f[5]) | (e4m3x2_rn_sat(f[6], f[7]) << 16);
    if (!POW2) {
      lo ^= 0x80808080u;
      hi ^= 0x80808080u;
    }
  } else if (S != 0.0f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) lo |= static_cast<uint32_t>(e4m3_rn_sat(f[i] / S)) << (8 * i);
#pragma unroll
    for (int i = 0; i < 4; ++i) hi |= static_cast<uint32_t>(e4m3_rn_sat(f[4 + i] / S)) << (8 * i);
  }
  return make_uint2(lo, hi);
}

// max(|a|, |b|) and max(|a|, |b|, |c|), NaN if one is
__device__ __forceinline__ float amax_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
  return r;
}
__device__ __forceinline__ float amax_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// A 128-channel tile's scale from its 16 lanes' maxima; NaN where the tile
// holds an infinity or a NaN.
template <bool POW2>
__device__ __forceinline__ float tile_scale(float am) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) am = amax_nan(am, __shfl_xor_sync(0xffffffffu, am, o));
  if (!(am <= 3.402823466e38f)) return __uint_as_float(0x7FFFFFFFu);
  if (POW2) return pow2_scale(am);
  // am / 448, correctly rounded: through 1 / 448 and one residual, by the
  // division where that could leave the normal range
  return am >= 0x1p-100f ? div_by_recip(am, 448.0f, 1.0f / 448.0f) : am / 448.0f;
}

// What is left of a chunk once rstd is known: y (stored as bf16 if y is given),
// the tile's scale, the codes.  Every lane of the warp calls it; `in`: the chunk
// is inside the row (a tile's 16 lanes all are, or none).  f: h, overwritten.
template <bool POW2>
__device__ __forceinline__ void finish_chunk(float (&f)[8], const float (&w)[8], float rstd, bool in,
                                             __nv_bfloat16 *y, uint8_t *q, float *s) {
  mul8(f, rstd);
  mul8(f, w);
  float am = 0.0f;
  if (in) {
    am = amax_nan(amax_nan(f[0], f[1], f[2]), amax_nan(f[3], f[4], f[5]), amax_nan(f[6], f[7]));
    if (y) store8(y, f);
  }
  const float S = tile_scale<POW2>(am);
  if (in) {
    *reinterpret_cast<uint2 *>(q) = tile_codes<POW2>(f, S);
    if ((threadIdx.x & 15) == 0) *s = S;
  }
}

// 1 / sqrt(ss / cols + eps): the hardware's reciprocal square root r of v and one
// Newton step r + r (1 - v r^2) / 2 with v r taken to twice FP32's digits, which
// leaves about half an FP32 step (1.0f / sqrtf(v) rounds twice).
__device__ __forceinline__ float rstd_of(float ss, int cols, float eps) {
  const float v = ss / static_cast<float>(cols) + eps;
  const float r = rsqrtf(v);
  if (!(v <= 3.402823466e38f)) return r;  // infinity gives 0, NaN itself
  const float p = v * r;
  const float h = fmaf(-fmaf(v, r, -p), r, fmaf(-p, r, 1.0f));
  return fmaf(0.5f * h, r, r);
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
  typename ChunkOf<TS>::type hc[CH];
  float ss = 0.0f;
  const TS *x = static_cast<const TS *>(p.x) + r * p.ld_x;
  const TS *rs = p.resid ? static_cast<const TS *>(p.resid) + r * p.ld_r : nullptr;
  // the weight: with one chunk a thread asked for with the row (few rows: its
  // latency would stand alone behind the row's sum), else where it is used
  auto weight = [&](int c, bool in, float (&w)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 1.0f;
    if (in && p.w) load8(p.w + c * 8, w);
  };
  float w0[8];
  if (CH == 1) weight(threadIdx.x, live && static_cast<int>(threadIdx.x) < nch, w0);
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int c = threadIdx.x + k * blockDim.x;
#pragma unroll
    for (int i = 0; i < 8; ++i) f[k][i] = 0.0f;
    if (live && c < nch) load_h<false>(x + c * 8, rs ? rs + c * 8 : nullptr, f[k], hc[k]);
    ss = sum_sq(f[k], ss);
  }
  ss = row_sum(ss, buf);
  const float rstd = rstd_of(ss, p.cols, p.eps);
  if (live && threadIdx.x == 0 && p.rstd) p.rstd[r] = rstd;
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int c = threadIdx.x + k * blockDim.x;
    const bool in = live && c < nch;
    float w[8];
    if (CH == 1) {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = w0[i];
    } else {
      weight(c, in, w);
    }
    if (in && p.h) store_h(static_cast<TS *>(p.h) + r * p.cols + c * 8, f[k], hc[k]);
    finish_chunk<POW2>(f[k], w, rstd, in, p.y ? p.y + r * p.cols + c * 8 : nullptr, p.q + r * p.cols + c * 8,
                       p.s + r * (p.cols / 128) + (c >> 4));
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

// Rows too long for the ring below: 4 chunks a thread, straight from memory.
template <typename TY, typename TS, typename TX, int CH>
__global__ void __launch_bounds__(1024, 1) add_rmsnorm_bwd_kernel(const NormBwd p) {
  __shared__ float buf[2][32];
  dependents_start();
  const int nch = p.cols / 8;
  float dw[CH][8];
#pragma unroll
  for (int k = 0; k < CH; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[k][i] = 0.0f;
  int ph = 0;
  for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x, ph ^= 1) {
    float n[CH][8], g[CH][8];
    float sum = 0.0f;
    const float rstd = p.rstd[r];
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = threadIdx.x + k * blockDim.x;
      if (c < nch) {
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
      if (c < nch) {
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
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int c = threadIdx.x + k * blockDim.x;
    if (c < nch) store8(p.dw_part + static_cast<int64_t>(blockIdx.x) * p.cols + c * 8, dw[k]);
  }
}

// ------------------------------------------------------ rows through a ring
// For batches that give each CTA several rows: a CTA stays and takes rows
// blockIdx.x, + gridDim.x, ...; one thread copies the next rows' inputs into a
// ring of shared-memory stages (bulk copies, one per input) while the CTA works
// on the current one.  Two 8-channel chunks per thread; the weight (and dw)
// stay in registers from row to row.  One barrier per row, for the row's sum:
// every thread has taken its inputs out of the stage by then, so the stage's
// next copy starts right behind it.
namespace {
constexpr int kRing = 4;  // stages at most
struct RingBars {
  uint64_t full[kRing];
  alignas(16) float red[2][32];
  int abort_flag;
};

// This thread of the CTA, over both dimensions.
__device__ __forceinline__ int tid() { return threadIdx.y * blockDim.x + threadIdx.x; }

// Sum over the threads of one row (threadIdx.x): each warp's sum into `red`, one
// barrier of the CTA, the row's warps' sums in a fixed order.  red's slots
// behind the CTA's warps stay zero.
__device__ __forceinline__ float ring_sum(float v, float *red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) red[tid() >> 5] = v;
  __syncthreads();
  const int nw = blockDim.x >> 5;
  float s = 0.0f;
  if (blockDim.y == 1) {
    for (int i = 0; i < nw; i += 4) {
      const float4 q = *reinterpret_cast<const float4 *>(red + i);
      s += (q.x + q.y) + (q.z + q.w);
    }
  } else {
    for (int i = 0; i < nw; ++i) s += red[threadIdx.y * nw + i];
  }
  return s;
}

__device__ __forceinline__ void ring_init(RingBars *b, int stages) {
  for (int i = tid(); i < 64; i += blockDim.x * blockDim.y) b->red[i >> 5][i & 31] = 0.0f;
  if (tid() == 0) {
    for (int i = 0; i < stages; ++i) mbar_init(&b->full[i], 1);
    b->abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
}

// Copies still in flight (only after a wait that gave up) land before the CTA
// leaves.
__device__ __forceinline__ void ring_drain(RingBars *b, int stages, uint32_t rows) {
  if (tid() == 0 && b->abort_flag) {
    int quiet = 0;
    const WaitCtl drain{&quiet, nullptr, 100000000ull};
    const uint32_t n = rows < static_cast<uint32_t>(stages) ? rows : stages;
    for (uint32_t i = rows - n; i < rows; ++i) mbar_wait(&b->full[i % stages], (i / stages) & 1, drain);
  }
  __syncthreads();
}
}  // namespace

template <typename TS, bool POW2, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) add_rmsnorm_quant_ring_kernel(const NormFwd p, int stages) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ __align__(16) RingBars bars;
  const int nch = p.cols / 8;
  const uint32_t in_bytes = static_cast<uint32_t>(p.cols * sizeof(TS));
  const uint32_t stage_bytes = p.resid ? 2 * in_bytes : in_bytes;
  ring_init(&bars, stages);
  const int64_t step = gridDim.x;
  auto copy_in = [&](uint32_t i) {
    const int64_t r = blockIdx.x + i * step;
    if (r >= p.rows) return;
    uint8_t *st = ring + (i % stages) * stage_bytes;
    uint64_t *bar = &bars.full[i % stages];
    mbar_arrive_expect_tx(bar, stage_bytes);
    bulk_load(st, static_cast<const TS *>(p.x) + r * p.ld_x, in_bytes, bar);
    if (p.resid) bulk_load(st + in_bytes, static_cast<const TS *>(p.resid) + r * p.ld_r, in_bytes, bar);
  };
  if (threadIdx.x == 0)
    for (int i = 0; i < stages; ++i) copy_in(i);
  float w[2][8];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int c = threadIdx.x + k * blockDim.x;
#pragma unroll
    for (int i = 0; i < 8; ++i) w[k][i] = 1.0f;
    if (p.w && c < nch) load8(p.w + c * 8, w[k]);
  }
  const WaitCtl ctl{&bars.abort_flag, nullptr, kDefaultWaitLimitNs};
  uint32_t it = 0;
  for (int64_t r = blockIdx.x; r < p.rows; r += step, ++it) {
    const int s = it % stages;
    const bool ok = mbar_wait(&bars.full[s], (it / stages) & 1, ctl);
    const TS *x = reinterpret_cast<const TS *>(ring + s * stage_bytes);
    float f[2][8], ss = 0.0f;
    typename ChunkOf<TS>::type hc[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int c = threadIdx.x + k * blockDim.x;
#pragma unroll
      for (int i = 0; i < 8; ++i) f[k][i] = 0.0f;
      if (c < nch) load_h<true>(x + c * 8, p.resid ? x + p.cols + c * 8 : nullptr, f[k], hc[k]);
      ss = sum_sq(f[k], ss);
    }
    ss = ring_sum(ss, bars.red[it & 1]);
    if (threadIdx.x == 0) copy_in(it + stages);
    float rstd = rstd_of(ss, p.cols, p.eps);
    if (!ok) rstd = __uint_as_float(0x7FFFFFFFu);  // a copy that never arrived shows as NaN
    if (threadIdx.x == 0 && p.rstd) p.rstd[r] = rstd;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int c = threadIdx.x + k * blockDim.x;
      const bool in = c < nch;
      if (in && p.h) store_h(static_cast<TS *>(p.h) + r * p.cols + c * 8, f[k], hc[k]);
      finish_chunk<POW2>(f[k], w[k], rstd, in, p.y ? p.y + r * p.cols + c * 8 : nullptr, p.q + r * p.cols + c * 8,
                         p.s + r * (p.cols / 128) + (c >> 4));
    }
  }
  ring_drain(&bars, stages, it);
}

// Backward.  blockDim = (threads per row, rows per stage): short rows go several
// to a stage (they are contiguous), each with its own warps.
template <typename TY, typename TS, typename TX, int MAXT>
__global__ void __launch_bounds__(MAXT, 1) add_rmsnorm_bwd_ring_kernel(const NormBwd p, int stages) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ __align__(16) RingBars bars;
  dependents_start();
  const int nch = p.cols / 8, nrow = blockDim.y, ty = threadIdx.y;
  const uint32_t y_bytes = static_cast<uint32_t>(p.cols * sizeof(TY)), s_bytes = static_cast<uint32_t>(p.cols * sizeof(TS));
  const uint32_t row_bytes = y_bytes + (p.dres ? 2 * s_bytes : s_bytes);
  const uint32_t h_off = nrow * y_bytes, d_off = h_off + nrow * s_bytes, stage_bytes = nrow * row_bytes;
  ring_init(&bars, stages);
  const int64_t step = static_cast<int64_t>(gridDim.x) * nrow, first = static_cast<int64_t>(blockIdx.x) * nrow;
  auto copy_in = [&](uint32_t i) {
    const int64_t r = first + i * step;
    if (r >= p.rows) return;
    const uint32_t n = p.rows - r < nrow ? static_cast<uint32_t>(p.rows - r) : nrow;
    uint8_t *st = ring + (i % stages) * stage_bytes;
    uint64_t *bar = &bars.full[i % stages];
    mbar_arrive_expect_tx(bar, n * row_bytes);
    bulk_load(st, static_cast<const TY *>(p.dy) + r * p.cols, n * y_bytes, bar);
    bulk_load(st + h_off, static_cast<const TS *>(p.h) + r * p.cols, n * s_bytes, bar);
    if (p.dres) bulk_load(st + d_off, static_cast<const TS *>(p.dres) + r * p.cols, n * s_bytes, bar);
  };
  if (tid() == 0)
    for (int i = 0; i < stages; ++i) copy_in(i);
  float w[2][8], dw[2][8];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int c = threadIdx.x + k * blockDim.x;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      w[k][i] = 1.0f;
      dw[k][i] = 0.0f;
    }
    if (p.w && c < nch) load8(p.w + c * 8, w[k]);
  }
  const WaitCtl ctl{&bars.abort_flag, nullptr, kDefaultWaitLimitNs};
  uint32_t it = 0;
  float next = first + ty < p.rows ? __ldg(p.rstd + first + ty) : 0.0f;
  for (int64_t r0 = first; r0 < p.rows; r0 += step, ++it) {
    const int64_t r = r0 + ty;
    const bool live = r < p.rows;
    float rstd = next;
    if (r + step < p.rows) next = __ldg(p.rstd + r + step);
    const int s = it % stages;
    // a copy that never arrived shows as NaN
    if (!mbar_wait(&bars.full[s], (it / stages) & 1, ctl)) rstd = __uint_as_float(0x7FFFFFFFu);
    const uint8_t *st = ring + s * stage_bytes;
    float n[2][8], g[2][8], d[2][8], sum = 0.0f;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int c = threadIdx.x + k * blockDim.x;
      if (live && c < nch) {
        load8_sh(reinterpret_cast<const TY *>(st + ty * y_bytes) + c * 8, g[k]);
        load8_sh(reinterpret_cast<const TS *>(st + h_off + ty * s_bytes) + c * 8, n[k]);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[k][i] = 0.0f;
        if (p.dres) load8_sh(reinterpret_cast<const TS *>(st + d_off + ty * s_bytes) + c * 8, d[k]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          n[k][i] *= rstd;
          dw[k][i] = fmaf(g[k][i], n[k][i], dw[k][i]);
          g[k][i] *= w[k][i];
          sum = fmaf(g[k][i], n[k][i], sum);
        }
      }
    }
    const float m = ring_sum(sum, bars.red[it & 1]) / static_cast<float>(p.cols);
    if (tid() == 0) copy_in(it + stages);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int c = threadIdx.x + k * blockDim.x;
      if (live && c < nch) {
#pragma unroll
        for (int i = 0; i < 8; ++i) d[k][i] = fmaf(rstd, fmaf(-n[k][i], m, g[k][i]), d[k][i]);
        store8(static_cast<TX *>(p.dx) + r * p.cols + c * 8, d[k]);
      }
    }
  }
  ring_drain(&bars, stages, it);
  if (!p.dw_part) return;
  float *part = p.dw_part + static_cast<int64_t>(blockIdx.x) * p.cols;
  if (nrow == 1) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int c = threadIdx.x + k * blockDim.x;
      if (c < nch) store8(part + c * 8, dw[k]);
    }
    return;
  }
  // the rows of the CTA in order, through the ring's memory (every copy into
  // it has landed and been read)
  float *sh = reinterpret_cast<float *>(ring);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int c = threadIdx.x + k * blockDim.x;
    if (c < nch) {
#pragma unroll
      for (int i = 0; i < 8; i += 4)
        *reinterpret_cast<float4 *>(sh + ty * p.cols + c * 8 + i) =
            make_float4(dw[k][i], dw[k][i + 1], dw[k][i + 2], dw[k][i + 3]);
    }
  }
  __syncthreads();
  for (int c = tid(); c < p.cols; c += blockDim.x * blockDim.y) {
    float t = 0.0f;
    for (int i = 0; i < nrow; ++i) t += sh[i * p.cols + c];
    part[c] = t;
  }
}

// dw[c] = sum over the parts, 32 columns per CTA: each of 32 warps takes every
// 32nd part, then the warps' sums are added in warp order.
__global__ void __launch_bounds__(1024) norm_dw_join_kernel(const float *part, int n_part, int cols, float *dw) {
  __shared__ float sh[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.0f;
  predecessor_done();
#pragma unroll 4
  for (int i = warp; i < n_part; i += 32) s += __ldcg(part + static_cast<int64_t>(i) * cols + c);
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

constexpr int kMaxCtas = 8;  // per SM
constexpr int kSmemPerSM = 233472 - 1024;  // shared memory of an SM, less one CTA's reserve

// How a ring kernel goes over `rows` rows of `row_bytes` inputs: threads per
// row, rows per stage, CTAs per SM, stages; ok = false where two stages do not
// fit or a thread would hold more than two chunks.  `threads_per_sm`: as many as
// the kernel's registers allow; `several`: short rows go several to a stage, up
// to 256 threads.
struct RingPlan {
  bool ok;
  int threads, nrow, per_sm, stages;
  int smem;
  int64_t grid;
};
inline RingPlan ring_plan(int64_t rows, int cols, int64_t row_bytes, int threads_per_sm, bool several) {
  RingPlan p{};
  p.threads = (cols / 16 + 31) / 32 * 32;
  if (p.threads > 1024) return p;
  p.nrow = several && p.threads <= 128 ? 256 / p.threads : 1;
  const int64_t bytes = row_bytes * p.nrow;
  int per_sm = threads_per_sm / (p.threads * p.nrow);
  if (per_sm > kMaxCtas) per_sm = kMaxCtas;
  if (per_sm < 1) per_sm = 1;
  // fewer CTAs, if that is what two stages take
  while (per_sm > 1 && (2 * bytes + 1536) * per_sm > kSmemPerSM) --per_sm;
  int64_t st = (kSmemPerSM / per_sm - 1536) / bytes;
  if (st > kRing) st = kRing;
  if (st < 2) return p;
  p.ok = true;
  p.per_sm = per_sm;
  p.stages = static_cast<int>(st);
  p.smem = static_cast<int>(st * bytes);
  const int64_t most = static_cast<int64_t>(moe_host::sm_count()) * per_sm, want = (rows + p.nrow - 1) / p.nrow;
  p.grid = want < most ? want : most;
  return p;
}

template <typename TS, int CH, bool POW2>
cudaError_t launch_norm_rows(const NormFwd &p, cudaStream_t st) {
  const dim3 b = norm_block(p.cols, CH);
  const unsigned grid = static_cast<unsigned>((p.rows + b.y - 1) / b.y);
  if constexpr (CH == 1) {  // (rows of several chunks a thread have more than 256 threads)
    if (b.x * b.y <= 256) {
      add_rmsnorm_quant_kernel<TS, CH, POW2, 256><<<grid, b, 0, st>>>(p);
      return cudaGetLastError();
    }
  }
  add_rmsnorm_quant_kernel<TS, CH, POW2, 1024><<<grid, b, 0, st>>>(p);
  return cudaGetLastError();
}

template <typename TS, bool POW2>
cudaError_t launch_norm_fwd(const NormFwd &p, cudaStream_t st) {
  const int64_t row_bytes = static_cast<int64_t>(p.cols) * sizeof(TS) * (p.resid ? 2 : 1);
  // The ring pays where a CTA gets several rows of some length (T = 16384, bf16:
  // 198 us against 329 at 7168 channels, 28 against 29 at 1024, 22 against 13 at
  // 512).
  const RingPlan pl = ring_plan(p.rows, p.cols, row_bytes, 1024, false);
  if (pl.ok && p.cols > 1024 && p.rows >= 2 * pl.grid) {
    if (pl.threads <= 512) {
      static std::atomic<uint64_t> done{0};
      if (const cudaError_t e = smem_attr_once(add_rmsnorm_quant_ring_kernel<TS, POW2, 512, 2>, kSmemPerSM - 1536, done))
        return e;
      add_rmsnorm_quant_ring_kernel<TS, POW2, 512, 2>
          <<<static_cast<unsigned>(pl.grid), pl.threads, pl.smem, st>>>(p, pl.stages);
    } else {
      static std::atomic<uint64_t> done{0};
      if (const cudaError_t e = smem_attr_once(add_rmsnorm_quant_ring_kernel<TS, POW2, 1024, 1>, kSmemPerSM - 1536, done))
        return e;
      add_rmsnorm_quant_ring_kernel<TS, POW2, 1024, 1>
          <<<static_cast<unsigned>(pl.grid), pl.threads, pl.smem, st>>>(p, pl.stages);
    }
    return cudaGetLastError();
  }
  // A row or two per CTA: as many threads as the row has chunks, up to 1024
  // (one token, 7168 channels: 8 us with one chunk a thread, 12 with four).
  return p.cols <= 8192 ? launch_norm_rows<TS, 1, POW2>(p, st) : launch_norm_rows<TS, 4, POW2>(p, st);
}

template <typename TY, typename TS>
int64_t bwd_row_bytes(int cols, bool dres) {
  return static_cast<int64_t>(cols) * (sizeof(TY) + sizeof(TS) * (dres ? 2 : 1));
}
constexpr int kCh = 4;  // chunks a thread in the rows kernel

template <typename TY, typename TS, typename TX>
cudaError_t launch_norm_bwd(const NormBwd &p, int *parts, cudaStream_t st) {
  const RingPlan pl = ring_plan(p.rows, p.cols, bwd_row_bytes<TY, TS>(p.cols, p.dres != nullptr), 512, true);
  if (pl.ok) {
    *parts = static_cast<int>(pl.grid);
    if (pl.threads <= 512) {
      static std::atomic<uint64_t> done{0};
      if (const cudaError_t e = smem_attr_once(add_rmsnorm_bwd_ring_kernel<TY, TS, TX, 512>, kSmemPerSM - 1536, done))
        return e;
      add_rmsnorm_bwd_ring_kernel<TY, TS, TX, 512>
          <<<static_cast<unsigned>(pl.grid), dim3(pl.threads, pl.nrow), pl.smem, st>>>(p, pl.stages);
    } else {
      static std::atomic<uint64_t> done{0};
      if (const cudaError_t e = smem_attr_once(add_rmsnorm_bwd_ring_kernel<TY, TS, TX, 1024>, kSmemPerSM - 1536, done))
        return e;
      add_rmsnorm_bwd_ring_kernel<TY, TS, TX, 1024>
          <<<static_cast<unsigned>(pl.grid), pl.threads, pl.smem, st>>>(p, pl.stages);
    }
    return cudaGetLastError();
  }
  // rows too long for two stages of the ring (above about 9000 FP32 channels)
  const int64_t most = 2 * static_cast<int64_t>(moe_host::sm_count());
  *parts = static_cast<int>(p.rows < most ? p.rows : most);
  add_rmsnorm_bwd_kernel<TY, TS, TX, kCh><<<*parts, dim3(norm_block(p.cols, kCh).x), 0, st>>>(p);  // a row a CTA
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

// An upper bound on the CTAs of either backward kernel.
int norm_bwd_parts(int64_t rows) {
  const int64_t most = kMaxCtas * static_cast<int64_t>(moe_host::sm_count());
  return static_cast<int>(rows < most ? rows : most);
}

cudaError_t launch_add_rmsnorm_bwd(const void *dy, bool dy_f32, const void *h, const void *dres, bool f32,
                                   const float *w, const float *rstd, int64_t rows, int cols, void *dx, bool dx_f32,
                                   float *dw, float *part, cudaStream_t st) {
  if (rows == 0) return dw ? cudaMemsetAsync(dw, 0, sizeof(float) * cols, st) : cudaSuccess;
  const NormBwd p{dy, h, dres, w, rstd, rows, cols, dx, dw ? part : nullptr};
  int n = 0;
  using B = __nv_bfloat16;
  cudaError_t e;
  if (dy_f32)
    e = f32 ? (dx_f32 ? launch_norm_bwd<float, float, float>(p, &n, st) : launch_norm_bwd<float, float, B>(p, &n, st))
            : (dx_f32 ? launch_norm_bwd<float, B, float>(p, &n, st) : launch_norm_bwd<float, B, B>(p, &n, st));
  else
    e = f32 ? (dx_f32 ? launch_norm_bwd<B, float, float>(p, &n, st) : launch_norm_bwd<B, float, B>(p, &n, st))
            : (dx_f32 ? launch_norm_bwd<B, B, float>(p, &n, st) : launch_norm_bwd<B, B, B>(p, &n, st));
  if (e != cudaSuccess || !dw) return e;
  return launch_next(norm_dw_join_kernel, dim3(static_cast<unsigned>(cols / 32)), dim3(1024), 0, st,
                     static_cast<const float *>(part), n, cols, dw);
}

}  // namespace moe
