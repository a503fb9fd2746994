// balance.cu -- sequence-wise balance loss and per-expert counts of packed
// sequences (its gradient is part of the router's backward, router_bwd.cu).
//
// "DeepSeek-V3 Technischer Bericht" (xyznot.com/de), Methode section 2, in the
// technical report's form.  For a sequence of L tokens:
//   c_i = picks of expert i,  f_i = N_r / (K_r L) c_i,
//   P_i = (1/L) sum_t s_{i,t} / sum_j s_{j,t},  loss = alpha sum_i f_i P_i.
// Bound by reading the logit partials once.  A sequence may be as long as the
// batch, so the tokens are cut into chunks that many CTAs take side by side; a
// CTA sums the pieces of the sequences inside its chunk (piece c + s for chunk
// c and sequence s: each chunk border and each sequence border starts a new
// one), and one CTA per sequence adds its pieces in token order.  The result
// does not depend on the schedule.
#include "common.cuh"
#include "kernels.h"
#include "operators.cuh"
#include "router_math.cuh"

namespace moe {

namespace {
constexpr int BAL_WARPS = 8;

struct BalArgs {
  const float *partial;
  int n_ks;
  int64_t T;
  int Nr, Kr;
  const int32_t *idx;
  const int32_t *off;
  int n_seq;
  int chunk;      // tokens per chunk
  int n_chunks;
  float *p_part;  // [n_chunks + n_seq, Nr] sums of the normalised affinities
  int32_t *c_part;  // [n_chunks + n_seq, Nr] picks
  int32_t *err;
};
}  // namespace

template <bool VEC, int B>
__global__ void __launch_bounds__(BAL_WARPS * 32, B == 1 ? 4 : 2) balance_pieces_kernel(const BalArgs a) {
  __shared__ __align__(16) float p_sh[BAL_WARPS][EPL * 32];
  __shared__ int c_sh[EPL * 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t c0 = static_cast<int64_t>(blockIdx.x) * a.chunk;
  const int64_t c1 = c0 + a.chunk < a.T ? c0 + a.chunk : a.T;
  dependents_start();
  bool bad = false;
  int64_t t0 = c0;
  while (t0 < c1) {  // every turn moves t0 forward, whatever the offsets hold
    const int s = seq_of(a.off, a.n_seq, t0, lane);
    if (s >= a.n_seq) break;
    if (a.off[s] > t0) {  // tokens before the first sequence belong to none
      t0 = a.off[s];
      continue;
    }
    const int64_t end = a.off[s + 1];
    if (end <= t0) break;  // only with wrong offsets
    const int64_t t1 = end < c1 ? end : c1;
    float acc[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) acc[i] = 0.0f;
    for (int i = threadIdx.x; i < EPL * 32; i += blockDim.x) c_sh[i] = 0;
    __syncthreads();
    for (int64_t t = t0 + warp; t < t1; t += BAL_WARPS) {
      int e = 0;
      if (lane < a.Kr) e = a.idx[t * a.Kr + lane];
      float v[EPL];
      load_logits<VEC, B>(a.partial, a.n_ks, a.T, a.Nr, t, lane, v);
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        float om;
        sigmoid_pair(v[i], v[i], om);
        if (lane_expert(lane, i) >= a.Nr) v[i] = 0.0f;
        sum += v[i];
      }
      sum = warp_sum(sum);
      const float inv = share_scale(sum);
#pragma unroll
      for (int i = 0; i < EPL; ++i) acc[i] = fmaf(v[i], inv, acc[i]);
      if (lane < a.Kr) {
        if (e >= 0 && e < a.Nr)
          atomicAdd(&c_sh[e], 1);
        else
          bad = true;
      }
    }
#pragma unroll
    for (int g = 0; g < 2; ++g)
      *reinterpret_cast<float4 *>(&p_sh[warp][g * 128 + lane * 4]) =
          make_float4(acc[4 * g], acc[4 * g + 1], acc[4 * g + 2], acc[4 * g + 3]);
    __syncthreads();
    const int64_t piece = static_cast<int64_t>(blockIdx.x) + s;
    for (int e = threadIdx.x; e < a.Nr; e += blockDim.x) {
      float p = 0.0f;
#pragma unroll
      for (int w = 0; w < BAL_WARPS; ++w) p += p_sh[w][e];
      a.p_part[piece * a.Nr + e] = p;
      a.c_part[piece * a.Nr + e] = c_sh[e];
    }
    __syncthreads();
    t0 = t1;
  }
  if (bad) atomicOr(a.err, MOE_DEVERR_BAD_INDEX);
}

// Eight CTAs (a cluster) per sequence, 32 experts each: one CTA alone would
// read a long sequence's pieces at one SM's share of the L2's rate (9.8 us for
// 13 sequences in 16384 tokens, 5.1 us so).  A thread adds every
// 64th piece of 4 experts; then the lanes, the warps and the CTAs' shares of
// the loss in a fixed order.
constexpr int BAL_CTAS = 8;
constexpr int BAL_JW = 16;  // warps

__global__ void __cluster_dims__(BAL_CTAS, 1, 1) __launch_bounds__(BAL_JW * 32)
    balance_join_kernel(const BalArgs a, float alpha, float *__restrict__ loss, int32_t *__restrict__ counts) {
  __shared__ float p_sh[BAL_JW][32];
  __shared__ int c_sh[BAL_JW][32];
  __shared__ float term;
  const int s = blockIdx.x / BAL_CTAS, rank = static_cast<int>(cluster_ctarank());
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int e0 = rank * 32 + (lane & 7) * 4;
  const int sl = warp * 4 + (lane >> 3);  // 64 slices
  predecessor_done();
  int64_t b0 = a.off[s], b1 = a.off[s + 1];
  if (b0 < 0 || b1 < b0 || b1 > a.T) {  // wrong offsets: reported, and read as an empty sequence
    if (rank == 0 && threadIdx.x == 0) atomicOr(a.err, MOE_DEVERR_BAD_INDEX);
    b0 = b1 = 0;
  }
  float p[4] = {0.f, 0.f, 0.f, 0.f};
  int c[4] = {0, 0, 0, 0};
  if (e0 < a.Nr && b1 > b0) {
    const int k0 = static_cast<int>(b0 / a.chunk), k1 = static_cast<int>((b1 - 1) / a.chunk);
    if (a.Nr % 4 == 0) {
#pragma unroll 4
      for (int k = k0 + sl; k <= k1; k += BAL_JW * 4) {
        const int64_t at = static_cast<int64_t>(k + s) * a.Nr + e0;
        const float4 pv = *reinterpret_cast<const float4 *>(a.p_part + at);
        const int4 cv = *reinterpret_cast<const int4 *>(a.c_part + at);
        p[0] += pv.x, p[1] += pv.y, p[2] += pv.z, p[3] += pv.w;
        c[0] += cv.x, c[1] += cv.y, c[2] += cv.z, c[3] += cv.w;
      }
    } else {
      for (int k = k0 + sl; k <= k1; k += BAL_JW * 4) {
        const int64_t at = static_cast<int64_t>(k + s) * a.Nr + e0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (e0 + j < a.Nr) {
            p[j] += a.p_part[at + j];
            c[j] += a.c_part[at + j];
          }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
#pragma unroll
    for (int o = 8; o < 32; o <<= 1) {
      p[j] += __shfl_xor_sync(0xffffffffu, p[j], o);
      c[j] += __shfl_xor_sync(0xffffffffu, c[j], o);
    }
    if (lane < 8) {
      p_sh[warp][lane * 4 + j] = p[j];
      c_sh[warp][lane * 4 + j] = c[j];
    }
  }
  __syncthreads();
  if (warp == 0) {
    const int e = rank * 32 + lane;
    float ps = 0.0f;
    int cs = 0;
#pragma unroll
    for (int w = 0; w < BAL_JW; ++w) {
      ps += p_sh[w][lane];
      cs += c_sh[w][lane];
    }
    if (e < a.Nr) counts[static_cast<int64_t>(s) * a.Nr + e] = cs;
    const float v = warp_sum(e < a.Nr ? static_cast<float>(cs) * ps : 0.0f);
    if (lane == 0) term = v;
  }
  cluster_sync_all();
  if (rank == 0 && threadIdx.x == 0) {
    float tot = 0.0f;
    for (int i = 0; i < BAL_CTAS; ++i) {
      float v;
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(mapa_shared(smem_u32(&term), i)) : "memory");
      tot += v;
    }
    const float L = static_cast<float>(b1 - b0);
    loss[s] = b1 > b0 ? alpha * (static_cast<float>(a.Nr) / (static_cast<float>(a.Kr) * L)) * (tot / L) : 0.0f;
  }
  cluster_sync_all();  // the shares stay readable until rank 0 has them
}

// Tokens per chunk: enough chunks for four CTAs on every SM, at least BAL_WARPS
// tokens each.
int balance_chunk(int64_t T) {
  const int64_t sms = moe_host::sm_count();
  int64_t c = (T + 4 * sms - 1) / (4 * sms);
  c = (c + BAL_WARPS - 1) / BAL_WARPS * BAL_WARPS;
  return static_cast<int>(c < BAL_WARPS ? BAL_WARPS : c);
}

int64_t balance_pieces(int64_t T, int64_t n_seq) {
  const int c = balance_chunk(T);
  return (T + c - 1) / c + n_seq;
}

cudaError_t launch_balance_loss(const float *partial, int n_ks, int64_t T, int Nr, int Kr, const int32_t *idx,
                                const int32_t *off, int n_seq, float alpha, float *p_part, int32_t *c_part,
                                float *loss, int32_t *counts, int32_t *err, cudaStream_t st) {
  if (n_seq == 0) return cudaSuccess;
  BalArgs a{};
  a.partial = partial;
  a.n_ks = n_ks;
  a.T = T;
  a.Nr = Nr;
  a.Kr = Kr;
  a.idx = idx;
  a.off = off;
  a.n_seq = n_seq;
  a.chunk = balance_chunk(T);
  a.n_chunks = static_cast<int>((T + a.chunk - 1) / a.chunk);
  a.p_part = p_part;
  a.c_part = c_part;
  a.err = err;
  if (T > 0) {
    auto kernel = Nr % 4 == 0 ? (n_ks < 4 ? balance_pieces_kernel<true, 1> : balance_pieces_kernel<true, 4>)
                              : (n_ks < 4 ? balance_pieces_kernel<false, 1> : balance_pieces_kernel<false, 4>);
    kernel<<<a.n_chunks, BAL_WARPS * 32, 0, st>>>(a);
  }
  if (const cudaError_t e = cudaGetLastError()) return e;
  return launch_next(balance_join_kernel, dim3(static_cast<unsigned>(BAL_CTAS) * n_seq), dim3(BAL_JW * 32), 0, st, a, alpha, loss, counts);
}

}  // namespace moe
