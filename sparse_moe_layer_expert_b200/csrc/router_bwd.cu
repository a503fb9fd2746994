// router_bwd.cu -- backward of the router: the gradient of the logits
// z = x . e_i from the gates and from the sequence-wise balance loss, and its
// two products, dx = dz W_r and dW_r = dz^T x.
//
// With s = sigmoid(z), the chosen experts' normalised affinities
// gh_k = s_k / sum_sel s (gate g_k = route_scale gh_k), a_k = g_k dL/dg_k, the
// shares p_i = s_i / sum_j s_j and the loss's load factors f_i (constants, as
// the picks are):
//   dz_k += (1 - s_k) (a_k - gh_k sum_j a_j)              (chosen experts)
//   dz_i += dloss alpha / L  p_i (1 - s_i) (f_i - sum_j f_j p_j)
// 1 - s is formed as sigmoid(-z), which keeps its digits where s is near 1.
//
// dz is FP32 and the other operand of both products bf16, so dz is split into
// three bf16 parts of 8 significand bits each (by truncation: the parts add up
// to dz's 24 bits) and each product runs on the tensor cores once per part
// into one FP32 accumulator: FP32-grade products at three bf16 passes.  Two
// parts, rounded to nearest, would leave 2^-16 of each term, 2.5e-6 of it in the
// root mean square, where FP32 sums of a few thousand terms lose less than 1e-6.
//
// Kernels:
//   router_dz_kernel   a warp per run of tokens: dz, written in FP32 (when asked
//                      for) and as parts [3][T][Np] bf16, Np = N_r rounded up
//                      to 64 (zeros behind N_r)
//   router_dx_kernel   256 tokens x 256 columns per pair of CTAs, a token tile's
//                      parts resident over its strips of W_r; A = the parts
//                      (K-major), B = W_r as it lies (N-major)
//   router_dwr_kernel  all experts x 256 columns of x per pair of CTAs over a
//                      range of tokens, so x is read once; both operands
//                      M/N-major (tokens are the slow index of both)
//   router_dx_dwr_kernel  both products at once, pairs of CTAs for each
//   dwr_join_kernel    adds the token ranges' partial sums in range order
// Each is launched by launch_next behind the one before it and reads what that
// one or an earlier one wrote only behind predecessor_done.
#include "common.cuh"
#include "kernels.h"
#include "operators.cuh"
#include "router_math.cuh"

namespace moe {

namespace {

// Shared-memory descriptor of an operand whose M (or N) index is contiguous:
// 128-byte rows of 64 bf16 (one K index each) with the 128-byte swizzle, 8-row
// groups 1024 bytes apart along K, and 64-element groups `group_bytes` apart
// along M (or N).  16 K rows further is 2048 bytes.
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t saddr, uint32_t group_bytes) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(group_bytes >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
         (static_cast<uint64_t>(2) << 61);
}
// instruction-descriptor bits: A (B) with M (N) contiguous
constexpr uint32_t kIdescAMn = 1u << 15;
constexpr uint32_t kIdescBMn = 1u << 16;

struct DzArgs {
  const float *partial;
  int n_ks;
  int64_t T;
  int Nr, Kr;
  float route_scale;
  const int32_t *idx;
  const float *dgate;            // [T, K_r] or null
  const float *gdot;             // [rows, n_dot] or null: a_k = sum of row pos[t, k]
  const int32_t *pos;
  int n_dot;
  const int32_t *off;            // null: no balance loss
  int n_seq;
  const int32_t *counts;
  const float *dloss;            // [n_seq] or null (ones)
  float alpha;
  float *dlogits;                // or null
  __nv_bfloat16 *parts;          // or null
  int Np;
  int run;  // tokens per warp
  int32_t *err;
};

// v = hi + mid + lo, each the leading 8 significand bits of what is left, as
// bf16 in the upper half of o[k]
__device__ __forceinline__ void split3(float v, uint32_t (&o)[3]) {
  const bool inf = (__float_as_uint(v) & 0x7FFFFFFFu) == 0x7F800000u;
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    o[k] = __float_as_uint(v) & 0xFFFF0000u;
    v = inf ? 0.0f : v - __uint_as_float(o[k]);
  }
}

}  // namespace

// A warp takes `run` consecutive tokens; the load factors f of the sequence it
// is in stay in registers from token to token.
template <bool VEC, int B>
__global__ void __launch_bounds__(256, B == 1 ? 4 : 2) router_dz_kernel(const DzArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t w = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int64_t t0 = w * a.run, t1 = t0 + a.run < a.T ? t0 + a.run : a.T;
  dependents_start();
  int seq = -1;           // sequence whose f is held
  int64_t seq_end = t0;   // look for a sequence at the first token
  float f[EPL], kk = 0.0f;
#pragma unroll
  for (int i = 0; i < EPL; ++i) f[i] = 0.0f;
  for (int64_t t = t0; t < t1; ++t) {
    float dz[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) dz[i] = 0.0f;
    // the slots' indices and gradients, asked for before they are needed (lane r: slot r)
    int e = -1;
    float w_k = 0.0f;
    if ((a.dgate || a.gdot) && lane < a.Kr) {
      e = a.idx[t * a.Kr + lane];
      if (a.dgate) w_k = a.dgate[t * a.Kr + lane];
    }
    if (a.off) {
      float z[EPL];
      load_logits<VEC, B>(a.partial, a.n_ks, a.T, a.Nr, t, lane, z);
      if (t >= seq_end) {
        const int s = seq_of(a.off, a.n_seq, t, lane);
        seq = -1;
        seq_end = a.T;
        if (s < a.n_seq) {
          const int64_t b0 = a.off[s], b1 = a.off[s + 1];
          if (b0 <= t) {
            seq = s;
            seq_end = b1;
            const float L = static_cast<float>(b1 - b0);
            const float fl = static_cast<float>(a.Nr) / (static_cast<float>(a.Kr) * L);
            kk = (a.dloss ? a.dloss[s] : 1.0f) * (a.alpha / L);
            const int32_t *cnt = a.counts + static_cast<int64_t>(s) * a.Nr;
#pragma unroll
            for (int i = 0; i < EPL; ++i)
              f[i] = lane_expert(lane, i) < a.Nr ? fl * static_cast<float>(cnt[lane_expert(lane, i)]) : 0.0f;
          } else {
            seq_end = b0;  // before the first sequence
          }
        }
      }
      if (seq >= 0) {
        float sum = 0.0f, fp = 0.0f, po[EPL];
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          float s, om;
          sigmoid_pair(z[i], s, om);
          if (lane_expert(lane, i) >= a.Nr) s = 0.0f;
          sum += s;
          fp = fmaf(f[i], s, fp);
          po[i] = s * om;
        }
        sum = warp_sum(sum);
        fp = warp_sum(fp);
        const float inv = share_scale(sum);
        // the share first: kk inv alone could overflow where the affinities are tiny
        const float kfp = kk * (fp * inv);
#pragma unroll
        for (int i = 0; i < EPL; ++i) dz[i] = po[i] * inv * fmaf(kk, f[i], -kfp);
      }
    }
    if (a.dgate || a.gdot) {
      float s = 0.0f, om = 0.0f;
      if (lane < a.Kr) {
        if (e < 0 || e >= a.Nr) {
          atomicOr(a.err, MOE_DEVERR_BAD_INDEX);
          e = -1;
        } else {
          sigmoid_pair(load_logit<B>(a.partial, a.n_ks, a.T, a.Nr, t, e), s, om);
        }
      }
      const float sum = warp_sum(s);
      const float gh = sum > 0.0f ? s / sum : 0.0f;
      if (a.gdot) {
        w_k = 0.0f;
        if (e >= 0) {
          const float *d = a.gdot + static_cast<int64_t>(a.pos[t * a.Kr + lane]) * a.n_dot;
          for (int j = 0; j < a.n_dot; ++j) w_k += d[j];
        }
      } else {
        w_k = e >= 0 ? a.route_scale * w_k * gh : 0.0f;  // a_k
      }
      const float tot = warp_sum(w_k);
      const float d = om * (w_k - gh * tot);
      for (int r = 0; r < a.Kr; ++r) {
        const int er = __shfl_sync(0xffffffffu, e, r);
        const float dr = __shfl_sync(0xffffffffu, d, r);
        if (er >= 0 && ((er & 127) >> 2) == lane) {
          const int at = (er >> 7) * 4 + (er & 3);
#pragma unroll
          for (int i = 0; i < EPL; ++i)
            if (i == at) dz[i] += dr;
        }
      }
    }
    if (a.dlogits) {
      float *row = a.dlogits + t * a.Nr;
      if (VEC && (reinterpret_cast<uintptr_t>(a.dlogits) & 15) == 0) {
#pragma unroll
        for (int g = 0; g < 2; ++g)
          if (g * 128 + lane * 4 < a.Nr)
            *reinterpret_cast<float4 *>(row + g * 128 + lane * 4) =
                make_float4(dz[4 * g], dz[4 * g + 1], dz[4 * g + 2], dz[4 * g + 3]);
      } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i)
          if (lane_expert(lane, i) < a.Nr) row[lane_expert(lane, i)] = dz[i];
      }
    }
    if (a.parts) {
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        if (g * 128 + lane * 4 < a.Np) {  // Np is a multiple of 64; dz is 0 behind N_r
          uint32_t p[4][3];
#pragma unroll
          for (int j = 0; j < 4; ++j) split3(dz[4 * g + j], p[j]);
#pragma unroll
          for (int k = 0; k < 3; ++k)
            *reinterpret_cast<uint2 *>(a.parts + (static_cast<int64_t>(k) * a.T + t) * a.Np + g * 128 + lane * 4) =
                make_uint2(__byte_perm(p[0][k], p[1][k], 0x7632), __byte_perm(p[2][k], p[3][k], 0x7632));
        }
      }
    }
  }
}

// ------------------------------------------------------ products, CTA pairs
// Both products run on pairs of CTAs (two SMs, tcgen05 cta_group::2): M = 256
// over the two CTAs, N = 256, each CTA holding half of A's rows and half of
// B's, so an MMA reads 64 bytes of shared memory a cycle and SM (96 on a
// single CTA's 128 x 256 tile) and the operands' arrival fits beside it.
namespace {
constexpr int kParts = 3;

__device__ __forceinline__ void umma_bf16_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                               uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 3D and 4D tiled loads whose completion counts on an mbarrier of either CTA
// of the pair (as tma_load_2d_pair).
__device__ __forceinline__ void tma_load_3d_pair(void *dst, const CUtensorMap *map, uint32_t bar_caddr, int32_t x,
                                                 int32_t y, int32_t z, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint "
      "[%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_caddr), "r"(x), "r"(y), "r"(z), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void tma_load_4d_pair(void *dst, const CUtensorMap *map, uint32_t bar_caddr, int32_t x,
                                                 int32_t y, int32_t z, int32_t w, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint "
      "[%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_caddr), "r"(x), "r"(y), "r"(z), "r"(w), "l"(policy)
      : "memory");
}

// A pair's run [u0, u1) of the launch's units, in order.  (At most 2^14 stages
// of 2^20 tokens times 128 strips of 32768 columns, times the pairs: 2^28.)
struct PairUnits {
  int u0, u1;
};
__host__ __device__ inline PairUnits pair_units(int pair, int pairs, int units) {
  return PairUnits{static_cast<int>(static_cast<uint32_t>(pair) * units / pairs),
                   static_cast<int>(static_cast<uint32_t>(pair + 1) * units / pairs)};
}

// --------------------------------------------------------------- dx = dz W_r
// Units (256-token tile, 256-column strip), tile-major; a pair takes a run of
// them.  The parts are three times the bytes of W_r's strip, so they are what
// stays: a token tile's parts (Np experts x 128 tokens x 3 in each CTA, 192 KB)
// stay in shared memory over its strips while W_r streams past in stages of 32
// experts (half a strip's columns in each CTA), 64 KB a unit against 192 KB the
// other way round (T = 4096, N_r = 256, H = 7168, alone on the device: 43 us that
// way, 39 us this, where the products take 28 us at the library's matrix rate and
// the output 30 us at the card's write rate).  The next tile's parts arrive as the
// current one's last pass over each 64-expert block ends.  The epilogue turns
// TMEM's rows so that four lanes store 128 contiguous bytes of a row (a row per
// thread took 64 cycles an instruction in the L1).
constexpr int X_STAGES = 4;
constexpr int X_THREADS = 320;        // warp 0 TMA, warp 1 MMA (even CTA), warps 2..9 epilogue
constexpr int X_AB = 128 * 128;       // 128 tokens x 64 experts, one part
constexpr int X_KB = 4;               // 64-expert blocks at most
constexpr int X_A = X_KB * kParts * X_AB;
constexpr int X_K = 32;               // experts per stage of W_r
constexpr int X_KPB = 64 / X_K;       // stages per 64-expert block
constexpr int X_BG = X_K * 128;       // 32 experts x 64 columns
constexpr int X_B = 2 * X_BG;         // this CTA's 128 columns
constexpr int X_SMEM = 1024 + X_A + X_STAGES * X_B + 256;
static_assert(X_SMEM <= 232448, "shared memory budget");

struct DxArgs {
  int64_t T;
  int n_strips, m_tiles, cols;  // H / 256 and T / 256, rounded up; H
  int kb;                       // Np / 64
  float *dx;
  int accumulate;
  int32_t *err;
  uint64_t limit_ns;
};

struct DxBars {
  uint64_t full[X_STAGES];   // even CTA: the stage of both CTAs has landed
  uint64_t empty[X_STAGES];  // each CTA: the MMAs have read the stage
  uint64_t afull[X_KB], aempty[X_KB];
  uint64_t tfull[2], tempty[2];
  uint64_t teardown;
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(DxBars) <= 256, "barrier block");

// 16 TMEM lanes x 32 columns: r[4 j + 2 i + k] of lane l is row l / 4 + 8 i,
// column 8 j + 2 (l mod 4) + k.
__device__ __forceinline__ void tmem_ld_16x256(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// Four lanes hold columns 2 j, 2 j + 1 (j the lane in its four) of blocks
// 0..3, block b in f[2 b], f[2 b + 1]; afterwards lane j holds the eight columns
// of block j in order.  Two exchanges, with the lane two and one away.
__device__ __forceinline__ void quad_transpose(float (&f)[8], int lane) {
  const bool up2 = lane & 2, up1 = lane & 1;
  // blocks (0, 1) <-> (2, 3): keep the half of the lane's own pair
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float got = __shfl_xor_sync(0xffffffffu, up2 ? f[i] : f[4 + i], 2);
    if (up2)
      f[i] = got;
    else
      f[4 + i] = got;
  }
  // now f[0..3] are the pair's blocks from lanes 0/1 of the four, f[4..7] from lanes 2/3
#pragma unroll
  for (int g = 0; g < 2; ++g) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float got = __shfl_xor_sync(0xffffffffu, up1 ? f[4 * g + k] : f[4 * g + 2 + k], 1);
      if (up1)
        f[4 * g + k] = got;
      else
        f[4 * g + 2 + k] = got;
    }
  }
}

// dx += v, one FP32 addition per element, in the L2 (T = 4096, H = 7168: dx added
// to 76 us, overwritten 41; reading dx a block or a unit ahead and storing the sums
// took 88 and 116).
__device__ __forceinline__ void red_add_v4(float *p, const float4 &v) {
  asm volatile("red.relaxed.gpu.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p), "f"(v.x), "f"(v.y), "f"(v.z),
               "f"(v.w)
               : "memory");
}
}  // namespace

// Pair `pair` of `pairs`.  The CTA may have more warps than X_THREADS.
__device__ __forceinline__ void dx_pair(const CUtensorMap &map_a, const CUtensorMap &map_w, const DxArgs &args,
                                        int pair, int pairs) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *sa = smem, *sb = sa + X_A;
  DxBars *bars = reinterpret_cast<DxBars *>(sb + X_STAGES * X_B);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  if (threadIdx.x == 0) {
    for (int i = 0; i < X_STAGES; ++i) {
      mbar_init(&bars->full[i], 2);  // each CTA's producer announces its bytes
      mbar_init(&bars->empty[i], 1);
    }
    for (int i = 0; i < X_KB; ++i) {
      mbar_init(&bars->afull[i], 2);
      mbar_init(&bars->aempty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->tfull[i], 1);
      mbar_init(&bars->tempty[i], 16);
    }
    mbar_init(&bars->teardown, 1);
    bars->abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_map(&map_a);
    tma_prefetch_map(&map_w);
  }
  if (warp == 1) {
    tmem_alloc_pair(&bars->tmem_base, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  volatile int *abortp = &bars->abort_flag;
  const WaitCtl ctl{abortp, args.err, args.limit_ns};
  const PairUnits pu = pair_units(pair, pairs, args.n_strips * args.m_tiles);
  const int nk = args.kb * X_KPB;  // stages per unit
  dependents_start();
  predecessor_done();

  if (warp == 0) {
    if (lane == 0) {
      const uint64_t pol = policy_evict_last();  // every tile reads W_r again
      uint32_t it = 0, na = 0;  // stages; token tiles
      int tile = -1;
      bool stop = false;
      for (int u = pu.u0; u < pu.u1 && !stop; ++u) {
        if (*abortp) break;
        const bool fresh = u / args.n_strips != tile;
        tile = u / args.n_strips;
        const int strip = u % args.n_strips;
        for (int k = 0; k < nk; ++k, ++it) {
          if (fresh && k % X_KPB == 0) {  // the first stage that reads this block of the tile's parts
            const int kb = k / X_KPB;
            if (!mbar_wait(&bars->aempty[kb], (na & 1) ^ 1, ctl)) {
              stop = true;
              break;
            }
            const uint32_t bar = mapa_shared(smem_u32(&bars->afull[kb]), 0);
            mbar_arrive_expect_tx_cluster(bar, kParts * X_AB);
            tma_load_4d_pair(sa + kb * kParts * X_AB, &map_a, bar, 0, tile * 256 + rank * 128, kb, 0,
                             pol);
          }
          const int s = it % X_STAGES;
          if (!mbar_wait(&bars->empty[s], ((it / X_STAGES) & 1) ^ 1, ctl)) {
            stop = true;
            break;
          }
          const uint32_t bar = mapa_shared(smem_u32(&bars->full[s]), 0);
          mbar_arrive_expect_tx_cluster(bar, X_B);
          tma_load_3d_pair(sb + s * X_B, &map_w, bar, 0, k * X_K, strip * 4 + rank * 2, pol);
        }
        if (fresh) ++na;
      }
      // the stages in flight are read before this CTA may exit
      int quiet = 0;
      const WaitCtl drain{&quiet, nullptr, 100000000ull};
      const uint32_t n_inflight = it < X_STAGES ? it : X_STAGES;
      for (uint32_t j = it - n_inflight; j < it; ++j) mbar_wait(&bars->empty[j % X_STAGES], (j / X_STAGES) & 1, drain);
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      uint32_t it = 0, tc = 0, na = 0;
      int tile = -1;
      bool stop = false;
      const uint32_t idesc = idesc_bf16_f32(256, 256) | kIdescBMn;
      for (int u = pu.u0; u < pu.u1 && !stop; ++u, ++tc) {
        if (*abortp) break;
        const bool fresh = u / args.n_strips != tile;
        tile = u / args.n_strips;
        const bool last = u + 1 < pu.u1 && (u + 1) / args.n_strips != tile;  // another token tile follows
        const uint32_t buf = tc & 1;
        if (!mbar_wait(&bars->tempty[buf], ((tc >> 1) & 1) ^ 1, ctl)) break;
        const uint32_t d = tmem + buf * 256;
        for (int k = 0; k < nk; ++k, ++it) {
          const int s = it % X_STAGES, kb = k / X_KPB;
          if ((fresh && k % X_KPB == 0 && !mbar_wait(&bars->afull[kb], na & 1, ctl)) ||
              !mbar_wait(&bars->full[s], (it / X_STAGES) & 1, ctl)) {
            stop = true;
            break;
          }
          tc_fence_after();
          const uint64_t da = sw128_kmajor_desc(smem_u32(sa + kb * kParts * X_AB)) + (k % X_KPB) * (X_K * 2 >> 4);
          const uint64_t db = sw128_mnmajor_desc(smem_u32(sb + s * X_B), X_BG);
#pragma unroll
          for (int q = 0; q < X_K / 16; ++q)
#pragma unroll
            for (int p = 0; p < kParts; ++p)
              umma_bf16_pair(d, da + p * (X_AB >> 4) + 2 * q, db + (2048 >> 4) * q, idesc,
                             (k > 0 || q > 0 || p > 0) ? 1u : 0u);
          umma_commit_pair(&bars->empty[s], 0x3);
          if (last && k % X_KPB == X_KPB - 1) umma_commit_pair(&bars->aempty[kb], 0x3);
        }
        umma_commit_pair(&bars->tfull[buf], 0x3);
        if (fresh) ++na;
      }
      int quiet = 0;
      const WaitCtl drain{&quiet, nullptr, 100000000ull};
      umma_commit_pair(&bars->teardown, 0x1);
      mbar_wait(&bars->teardown, 0, drain);
    }
  } else if (warp < X_THREADS / 32) {
    const int q = warp & 3;           // TMEM lane quarter
    const int half = (warp - 2) >> 2;  // column half
    const bool wide = (reinterpret_cast<uintptr_t>(args.dx) & 31) == 0;
    uint32_t tc = 0;
    for (int u = pu.u0; u < pu.u1; ++u, ++tc) {
      const uint32_t buf = tc & 1;
      if (!mbar_wait(&bars->tfull[buf], (tc >> 1) & 1, ctl)) break;
      tc_fence_after();
      const int64_t t0 = static_cast<int64_t>(u / args.n_strips) * 256 + rank * 128 + q * 32;
      const int x0 = (u % args.n_strips) * 256 + half * 128;
      const uint32_t ta = tmem + (static_cast<uint32_t>(q * 32) << 16) + buf * 256 + half * 128;
      // H is a multiple of 128: a column half is in or out
#pragma unroll 1
      for (int c = 0; c < 4 && x0 < args.cols; ++c) {
        // 16 rows at a time: lane 4 i + j gets rows i and i + 8, columns 2 j and
        // 2 j + 1 of each of the four 8-column blocks; turned within each four
        // lanes so that lane j has block j whole, 32 bytes
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t v[16];
          tmem_ld_16x256(ta + c * 32 + (h << 20), v);
          tmem_ld_wait();
#pragma unroll
          for (int r8 = 0; r8 < 2; ++r8) {
            float f[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              f[2 * j] = __uint_as_float(v[4 * j + 2 * r8]);
              f[2 * j + 1] = __uint_as_float(v[4 * j + 2 * r8 + 1]);
            }
            quad_transpose(f, lane);
            const int64_t t = t0 + h * 16 + r8 * 8 + (lane >> 2);
            if (t < args.T) {
              float *dst = args.dx + t * args.cols + x0 + c * 32 + (lane & 3) * 8;
              if (args.accumulate) {
                red_add_v4(dst, make_float4(f[0], f[1], f[2], f[3]));
                red_add_v4(dst + 4, make_float4(f[4], f[5], f[6], f[7]));
              } else if (wide) {
                st_f32x8(dst, f);
              } else {
                reinterpret_cast<float4 *>(dst)[0] = make_float4(f[0], f[1], f[2], f[3]);
                reinterpret_cast<float4 *>(dst)[1] = make_float4(f[4], f[5], f[6], f[7]);
              }
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&bars->tempty[buf]), 0));
    }
  }
  // neither CTA leaves (or frees TMEM) while the other still works with its
  // shared memory, barriers or TMEM
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(X_THREADS, 1)
    router_dx_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_w,
                     const DxArgs args) {
  dx_pair(map_a, map_w, args, blockIdx.x >> 1, gridDim.x >> 1);
}

// ------------------------------------------------------------ dW_r = dz^T x
// Units (256-column strip of x, 64-token stage), strip-major, in as many equal runs
// as the device has pairs; a pair takes one run, or where dx's pairs have
// the other half of the SMs, two.  A strip's tokens are so shared out over several
// runs and every SM has the same work.  The tensor core's FP32 accumulation drops the bits
// below its 24 at every step (measured: the error grows with the number of
// steps, to 6e-6 of the result over 3300 tokens), so one TMEM accumulator takes
// WR_CHUNK stages (24 steps) at most: the epilogue warps add it into FP32
// registers while the next chunk's MMAs fill the other buffer.  At the end of a
// strip's run the registers go to the partial sums, piece (run + strip).
// A stage is two loads, one 4D box of the parts and one 3D box of x: as eight
// 2D boxes of 32 tokens each load cost about 110 ns and set the pace.
namespace {
constexpr int WR_THREADS = 384;              // warp 0 TMA, warp 1 MMA (even CTA), warps 4..11 epilogue
constexpr int WR_STAGES = 3;
constexpr int WR_TOK = 64;                   // tokens (K) per stage
constexpr int WR_CHUNK = 2;                  // stages per TMEM accumulation
constexpr int WR_G = WR_TOK * 128;           // 64 tokens x 64 experts (or columns)
constexpr int WR_A = kParts * 2 * WR_G;      // this CTA's 128 experts
constexpr int WR_B = 2 * WR_G;               // this CTA's 128 columns
constexpr int WR_STAGE = WR_A + WR_B;
constexpr int WR_SMEM = 1024 + WR_STAGES * WR_STAGE + 256;
static_assert(WR_SMEM <= 232448, "shared memory budget");

// A pair's run [u, end) of one strip, and how its stages fall into chunks: the
// MMA issuer and the epilogue walk it alike.
__device__ __forceinline__ int run_end(int u, int u1, int per_strip) {
  const int e = (u / per_strip + 1) * per_strip;
  return e < u1 ? e : u1;
}

struct DwrArgs {
  int64_t T;
  int n_strips, n_stages;  // H / 256 and T / 64, rounded up
  int Nr;
  int n_runs;              // what the units are shared out to
  float *part;             // [n_runs + n_strips, 256, 256]
  int32_t *err;
  uint64_t limit_ns;
};

struct DwrBars {
  uint64_t full[WR_STAGES];
  uint64_t empty[WR_STAGES];
  uint64_t tfull[2], tempty[2];
  uint64_t teardown;
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(DwrBars) <= 256, "barrier block");
}  // namespace

// Pair `pair` of `pairs` (WR_THREADS threads a CTA, launched with 168 registers each).
__device__ __forceinline__ void dwr_pair(const CUtensorMap &map_a, const CUtensorMap &map_x, const DwrArgs &args,
                                         int pair, int pairs) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  DwrBars *bars = reinterpret_cast<DwrBars *>(smem + WR_STAGES * WR_STAGE);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  if (threadIdx.x == 0) {
    for (int i = 0; i < WR_STAGES; ++i) {
      mbar_init(&bars->full[i], 2);
      mbar_init(&bars->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->tfull[i], 1);
      mbar_init(&bars->tempty[i], 16);
    }
    mbar_init(&bars->teardown, 1);
    bars->abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_map(&map_a);
    tma_prefetch_map(&map_x);
  }
  if (warp == 1) {
    tmem_alloc_pair(&bars->tmem_base, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  volatile int *abortp = &bars->abort_flag;
  const WaitCtl ctl{abortp, args.err, args.limit_ns};
  // this pair's share [r0, r1) of the runs that the units fall into
  const PairUnits runs = pair_units(pair, pairs, args.n_runs);
  const int units = args.n_strips * args.n_stages;

  dependents_start();
  predecessor_done();

  // Register split as in gemm_pair.cu: 128 * 72 + 256 * 216 = 384 * 168
  if (warp < 4) {
    setmaxnreg_dec<72>();
    if (warp == 0) {
      if (lane == 0) {
        const uint64_t pol_a = policy_evict_last();   // every strip reads the parts again
        const uint64_t pol_x = policy_evict_first();  // x is read once
        uint32_t it = 0;
        // the runs follow each other: one range of units
        const int u1 = runs.u1 > runs.u0 ? pair_units(runs.u1 - 1, args.n_runs, units).u1 : 0;
        for (int u = pair_units(runs.u0, args.n_runs, units).u0; u < u1; ++u, ++it) {
          const int s = it % WR_STAGES;
          if (*abortp || !mbar_wait(&bars->empty[s], ((it / WR_STAGES) & 1) ^ 1, ctl)) break;
          uint8_t *st = smem + s * WR_STAGE;
          const uint32_t bar = mapa_shared(smem_u32(&bars->full[s]), 0);
          const int t0 = (u % args.n_stages) * WR_TOK;
          mbar_arrive_expect_tx_cluster(bar, WR_STAGE);
          tma_load_3d_pair(st + WR_A, &map_x, bar, 0, t0, (u / args.n_stages) * 4 + rank * 2, pol_x);
          tma_load_4d_pair(st, &map_a, bar, 0, t0, rank * 2, 0, pol_a);
        }
        int quiet = 0;
        const WaitCtl drain{&quiet, nullptr, 100000000ull};
        const uint32_t n_inflight = it < WR_STAGES ? it : WR_STAGES;
        for (uint32_t j = it - n_inflight; j < it; ++j)
          mbar_wait(&bars->empty[j % WR_STAGES], (j / WR_STAGES) & 1, drain);
      }
    } else if (warp == 1) {
      if (lane == 0 && rank == 0) {
        uint32_t it = 0, tc = 0;
        bool stop = false;
        const uint32_t idesc = idesc_bf16_f32(256, 256) | kIdescAMn | kIdescBMn;
        for (int run = runs.u0; run < runs.u1 && !stop; ++run) {
          const PairUnits pu = pair_units(run, args.n_runs, units);
          for (int u = pu.u0; u < pu.u1 && !stop;) {
            const int end = run_end(u, pu.u1, args.n_stages);
            for (; u < end && !stop; ++tc) {
              const uint32_t buf = tc & 1;
              if (*abortp || !mbar_wait(&bars->tempty[buf], ((tc >> 1) & 1) ^ 1, ctl)) {
                stop = true;
                break;
              }
              const uint32_t d = tmem + buf * 256;
              for (int k = 0; k < WR_CHUNK && u < end; ++k, ++u, ++it) {
                const int s = it % WR_STAGES;
                if (!mbar_wait(&bars->full[s], (it / WR_STAGES) & 1, ctl)) {
                  stop = true;
                  break;
                }
                tc_fence_after();
                const uint32_t st = smem_u32(smem + s * WR_STAGE);
#pragma unroll
                for (int q = 0; q < WR_TOK / 16; ++q) {
                  const uint64_t db = sw128_mnmajor_desc(st + WR_A + q * 2048, WR_G);
#pragma unroll
                  for (int p = 0; p < kParts; ++p)
                    umma_bf16_pair(d, sw128_mnmajor_desc(st + p * 2 * WR_G + q * 2048, WR_G), db, idesc,
                                   (k > 0 || q > 0 || p > 0) ? 1u : 0u);
                }
                umma_commit_pair(&bars->empty[s], 0x3);
              }
              umma_commit_pair(&bars->tfull[buf], 0x3);
            }
          }
        }
        int quiet = 0;
        const WaitCtl drain{&quiet, nullptr, 100000000ull};
        umma_commit_pair(&bars->teardown, 0x1);
        mbar_wait(&bars->teardown, 0, drain);
      }
    }
  } else {
    setmaxnreg_inc<216>();
    const int q = warp & 3;
    const int wg = (warp - 4) >> 2;
    const bool live = rank * 128 + q * 32 < args.Nr;     // any expert in this warp
    uint32_t tc = 0;
    bool stop = false;
    for (int run = runs.u0; run < runs.u1 && !stop; ++run) {
      const PairUnits pu = pair_units(run, args.n_runs, units);
      for (int u = pu.u0; u < pu.u1 && !stop;) {
        const int strip = u / args.n_stages;
        const int end = run_end(u, pu.u1, args.n_stages);
        // 16-row halves h, 32-column blocks c: lane 4 i + j holds rows i, i + 8 and
        // columns 2 j, 2 j + 1 of each 8-column block (tmem_ld_16x256)
        float acc[2][4][16];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int j = 0; j < 16; ++j) acc[h][c][j] = 0.0f;
        for (; u < end; u += WR_CHUNK, ++tc) {
          const uint32_t buf = tc & 1;
          if (!mbar_wait(&bars->tfull[buf], (tc >> 1) & 1, ctl)) {
            stop = true;
            break;
          }
          if (live) {
            tc_fence_after();
            const uint32_t ta = tmem + (static_cast<uint32_t>(q * 32) << 16) + buf * 256 + wg * 128;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t v[2][16];
              tmem_ld_16x256(ta + c * 32, v[0]);
              tmem_ld_16x256(ta + c * 32 + (1 << 20), v[1]);
              tmem_ld_wait();
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < 16; ++j) acc[h][c][j] += __uint_as_float(v[h][j]);
            }
            tc_fence_before();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&bars->tempty[buf]), 0));
        }
        if (live) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int r8 = 0; r8 < 2; ++r8) {
              const int row = rank * 128 + q * 32 + h * 16 + r8 * 8 + (lane >> 2);  // expert
              float *o = args.part + (static_cast<int64_t>(run + strip) * 256 + row) * 256 + wg * 128 + (lane & 3) * 8;
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                float f[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  f[2 * j] = acc[h][c][4 * j + 2 * r8];
                  f[2 * j + 1] = acc[h][c][4 * j + 2 * r8 + 1];
                }
                quad_transpose(f, lane);
                if (row < args.Nr) st_f32x8(o + c * 32, f);
              }
            }
        }
        u = end;
      }
    }
  }
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(WR_THREADS, 1)
    router_dwr_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_x,
                      const DwrArgs args) {
  dwr_pair(map_a, map_x, args, blockIdx.x >> 1, gridDim.x >> 1);
}

// Both products side by side, the first dx_pairs pairs on dx.  One launch, so
// that both start behind router_dz_kernel by the same predecessor_done (dW_r as a
// launch of its own would have to wait for dx, or read dz without waiting).
constexpr int BOTH_SMEM = X_SMEM > WR_SMEM ? X_SMEM : WR_SMEM;
static_assert(X_THREADS <= WR_THREADS, "dx's warps");
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(WR_THREADS, 1)
    router_dx_dwr_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_w,
                         const DxArgs dx, const __grid_constant__ CUtensorMap map_b,
                         const __grid_constant__ CUtensorMap map_x, const DwrArgs dwr, int dx_pairs) {
  const int pair = blockIdx.x >> 1;
  if (pair < dx_pairs)
    dx_pair(map_a, map_w, dx, pair, dx_pairs);
  else
    dwr_pair(map_b, map_x, dwr, pair - dx_pairs, (gridDim.x >> 1) - dx_pairs);
}

// dW_r [Nr, cols] from the pieces of each strip, in token order.  CTA (4
// experts, strip): 64 threads of 4 columns for each expert.  A strip has
// runs / n_strips + 2 pieces at most; four are read at once.
__global__ void __launch_bounds__(256) dwr_join_kernel(const float *part, int pairs, int n_strips, int n_stages,
                                                        int Nr, int cols, float *out) {
  const int strip = blockIdx.y;
  const int e = blockIdx.x * 4 + (threadIdx.x >> 6), c = (threadIdx.x & 63) * 4;
  const int units = n_strips * n_stages;
  const int a = strip * n_stages, b = a + n_stages;  // the strip's units
  // the first pair whose run ends behind a, and the first that starts at or behind b
  int p0 = static_cast<int>(static_cast<uint32_t>(a) * pairs / units), p1 = p0;
  while (pair_units(p0, pairs, units).u1 <= a) ++p0;
  p1 = p0;
  while (p1 < pairs && pair_units(p1, pairs, units).u0 < b) ++p1;
  predecessor_done();
  if (e >= Nr || strip * 256 + c >= cols) return;
  const float *src = part + (static_cast<int64_t>(p0 + strip) * 256 + e) * 256 + c;
  const int n = p1 - p0;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = 0; i < n; i += 4) {
    float4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i + k < n) v[k] = __ldcg(reinterpret_cast<const float4 *>(src + (i + k) * 65536ll));
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i + k < n) {
        s.x += v[k].x;
        s.y += v[k].y;
        s.z += v[k].z;
        s.w += v[k].w;
      }
  }
  *reinterpret_cast<float4 *>(out + static_cast<int64_t>(e) * cols + strip * 256 + c) = s;
}

// -------------------------------------------------------------------- host
int router_parts_pitch(int Nr) { return (Nr + 63) / 64 * 64; }


namespace {
// Pairs of CTAs at most (one CTA per SM); a launch takes as many as are
// resident at once.
int64_t most_pairs() { return moe_host::sm_count() / 2; }

int dwr_stages(int64_t T) { return static_cast<int>((T + WR_TOK - 1) / WR_TOK); }
int strips_of(int cols) { return (cols + 255) / 256; }

int dwr_pairs(int64_t T, int cols) {
  const int64_t units = static_cast<int64_t>(strips_of(cols)) * dwr_stages(T);
  return static_cast<int>(units < most_pairs() ? units : most_pairs());
}
}  // namespace

// Whether dx and dW_r, both asked for, run side by side on half of the SMs each:
// dx alone is held up by its stores and dW_r by its loads, but with many units a
// pair both reach their own limit by themselves, the matrix rate or, with 64 experts
// and fewer (a third of the matrix work or less beside the same memory traffic),
// the memory's, which comes sooner.  (us a pass, one after the other / side by side,
// H = 7168: N_r = 256, T = 512 34.7 / 27.1, 2048 55.4 / 47.2, 4096 80.1 / 77.2,
// 8192 150.5 / 151.3, 16381 294 / 301; 128, 4096 69.7 / 68.6, 8192 125 / 127;
// 64, 2048 44.3 / 40.9, 4096 63.7 / 65.7, 8192 106 / 119.  H = 2048, 64 experts:
// 8192 49.8 / 47.9, 12288 65.4 / 64.8, 16381 77.6 / 82.0.)
static bool share_sms(int64_t T, int cols, int Nr) {
  const int64_t units = static_cast<int64_t>(strips_of(cols)) * ((T + 255) / 256);
  return units < (Nr > 64 ? 12 : 5) * most_pairs();
}

size_t router_dwr_scratch(int64_t T, int cols) {
  return T == 0 ? 0 : static_cast<size_t>(dwr_pairs(T, cols) + strips_of(cols)) * 256 * 256 * sizeof(float);
}

cudaError_t launch_router_dz(const RouterBwd &g, cudaStream_t st) {
  if (g.T == 0) return cudaSuccess;
  DzArgs a{};
  a.partial = g.partial;
  a.n_ks = g.n_ks;
  a.T = g.T;
  a.Nr = g.Nr;
  a.Kr = g.Kr;
  a.route_scale = g.route_scale;
  a.idx = g.idx;
  a.dgate = g.dgate;
  a.gdot = g.gdot;
  a.pos = g.pos;
  a.n_dot = g.n_dot;
  a.off = g.off;
  a.n_seq = g.n_seq;
  a.counts = g.counts;
  a.dloss = g.dloss;
  a.alpha = g.alpha;
  a.dlogits = g.dlogits;
  a.parts = static_cast<__nv_bfloat16 *>(g.parts);
  a.Np = router_parts_pitch(g.Nr);
  a.err = g.err;
  // as many warps as are resident at once (four CTAs on every SM)
  const int64_t warps = static_cast<int64_t>(moe_host::sm_count()) * 32;
  const int64_t run = (g.T + warps - 1) / warps;
  a.run = static_cast<int>(run < 8 ? run : 8);
  const unsigned grid = static_cast<unsigned>(((g.T + a.run - 1) / a.run + 7) / 8);
  auto kernel = g.Nr % 4 == 0 ? (g.n_ks < 4 ? router_dz_kernel<true, 1> : router_dz_kernel<true, 4>)
                              : (g.n_ks < 4 ? router_dz_kernel<false, 1> : router_dz_kernel<false, 4>);
  kernel<<<grid, 256, 0, st>>>(a);
  return cudaGetLastError();
}

// dx = dz W_r and dW_r = dz^T x, those asked for, behind launch_router_dz.
cudaError_t launch_router_products(const RouterProducts &g, cudaStream_t st) {
  if (g.T == 0)
    return g.dwr ? cudaMemsetAsync(g.dwr, 0, sizeof(float) * g.Nr * static_cast<size_t>(g.H), st) : cudaSuccess;
  const uint64_t Np = router_parts_pitch(g.Nr), t = g.T, h = g.H;
  // every operand in groups of 64 elements (128 bytes) of a row: parts [3][Np / 64][T][64], W_r [H / 64][Nr][64],
  // x [H / 64][T][64]
  const uint64_t dp[4] = {64, t, Np / 64, kParts}, sp[3] = {Np * 2, 128, t * Np * 2};
  const auto BF16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  static std::atomic<int> resident[3][64];
  DxArgs a{};
  CUtensorMap ma, mw;
  int64_t pairs = 0;
  if (g.dx) {
    const uint64_t dw[3] = {64, static_cast<uint64_t>(g.Nr), h / 64}, sw[2] = {h * 2, 128};
    const uint32_t ba[4] = {64, 128, 1, kParts}, bw[3] = {64, X_K, 2};
    if (moe_host::encode_tmap(&ma, BF16, g.parts, 4, dp, sp, ba) != 0 ||
        moe_host::encode_tmap(&mw, BF16, g.wr, 3, dw, sw, bw) != 0)
      return cudaErrorInvalidValue;
    a.T = g.T;
    a.cols = g.H;
    a.n_strips = strips_of(g.H);
    a.m_tiles = static_cast<int>((g.T + 255) / 256);
    a.kb = static_cast<int>(Np / 64);
    a.dx = g.dx;
    a.accumulate = g.accumulate;
    a.err = g.err;
    a.limit_ns = g.limit_ns;
    static std::atomic<uint64_t> done{0};
    if (const cudaError_t e = smem_attr_once(router_dx_kernel, X_SMEM, done)) return e;
    pairs = resident_pairs(router_dx_kernel, X_THREADS, X_SMEM, most_pairs(), resident[0]);
  }
  const int64_t units = static_cast<int64_t>(a.n_strips) * a.m_tiles;
  DwrArgs b{};
  CUtensorMap mb, mx;
  if (g.dwr) {
    const uint64_t dx[3] = {64, t, h / 64}, sx[2] = {h * 2, 128};
    const uint32_t bb[4] = {64, WR_TOK, 2, kParts}, bx[3] = {64, WR_TOK, 2};
    if (moe_host::encode_tmap(&mb, BF16, g.parts, 4, dp, sp, bb) != 0 ||
        moe_host::encode_tmap(&mx, BF16, g.x, 3, dx, sx, bx) != 0)
      return cudaErrorInvalidValue;
    b.T = g.T;
    b.n_strips = strips_of(g.H);
    b.n_stages = dwr_stages(g.T);
    b.Nr = g.Nr;
    b.part = g.part;
    b.err = g.err;
    b.limit_ns = g.limit_ns;
    static std::atomic<uint64_t> done{0};
    if (const cudaError_t e = smem_attr_once(router_dwr_kernel, WR_SMEM, done)) return e;
    // the runs, and so the sums' order, are the same with and without dx beside them
    int64_t runs = resident_pairs(router_dwr_kernel, WR_THREADS, WR_SMEM, most_pairs(), resident[1]);
    if (runs > dwr_pairs(g.T, g.H)) runs = dwr_pairs(g.T, g.H);
    b.n_runs = static_cast<int>(runs);
  }
  if ((g.dx && pairs < 1) || (g.dwr && b.n_runs < 1)) return cudaErrorLaunchOutOfResources;

  cudaError_t e = cudaSuccess;
  if (g.dx && g.dwr && share_sms(g.T, g.H, g.Nr)) {
    static std::atomic<uint64_t> done{0};
    if ((e = smem_attr_once(router_dx_dwr_kernel, BOTH_SMEM, done)) != cudaSuccess) return e;
    const int64_t all = resident_pairs(router_dx_dwr_kernel, WR_THREADS, BOTH_SMEM, most_pairs(), resident[2]);
    int64_t p = (all + 1) / 2;
    if (p > units) p = units;
    // dW_r: a pair for each run where that many are left, else half as many
    const int64_t q = b.n_runs <= all - p ? b.n_runs : (b.n_runs + 1) / 2;
    e = launch_next(router_dx_dwr_kernel, dim3(static_cast<unsigned>(2 * (p + q))), dim3(WR_THREADS), BOTH_SMEM, st, ma,
                    mw, a, mb, mx, b, static_cast<int>(p));
  } else {
    if (g.dx)
      e = launch_next(router_dx_kernel, dim3(static_cast<unsigned>(2 * (pairs < units ? pairs : units))),
                      dim3(X_THREADS), X_SMEM, st, ma, mw, a);
    if (e == cudaSuccess && g.dwr)
      e = launch_next(router_dwr_kernel, dim3(static_cast<unsigned>(2 * b.n_runs)), dim3(WR_THREADS), WR_SMEM, st, mb, mx,
                      b);
  }
  if (e != cudaSuccess || !g.dwr) return e;
  return launch_next(dwr_join_kernel, dim3(static_cast<unsigned>((g.Nr + 3) / 4), static_cast<unsigned>(b.n_strips)),
                     dim3(256), 0, st, static_cast<const float *>(g.part), b.n_runs, b.n_strips, b.n_stages, g.Nr, g.H,
                     g.dwr);
}

}  // namespace moe
