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
// parts would leave an error of 2^-17 of each term.
//
// Kernels:
//   router_dz_kernel   one warp per token: dz, written in FP32 (when asked
//                      for) and as parts [3][T][Np] bf16, Np = N_r rounded up
//                      to 64 (zeros behind N_r)
//   router_dx_kernel   persistent over 128-token tiles of one 256-column strip
//                      of W_r, which stays in shared memory (K = Np <= 256);
//                      A = the parts (K-major), B = W_r as it lies (N-major)
//   router_dwr_kernel  all experts x 256 columns of x per CTA over a range of
//                      tokens, so x is read once; both operands M/N-major
//                      (tokens are the slow index of both)
//   dwr_join_kernel    adds the token ranges' partial sums in range order
#include "common.cuh"
#include "kernels.h"
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

__device__ __forceinline__ void tma_reduce_add_2d(const CUtensorMap *map, const void *src, int32_t x, int32_t y) {
  asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(smem_u32(src)), "r"(x), "r"(y)
               : "memory");
}

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
  int32_t *err;
};

// v = hi + mid + lo, each the leading 8 significand bits of what is left
__device__ __forceinline__ void split3(float v, __nv_bfloat16 (&o)[3]) {
  const bool inf = (__float_as_uint(v) & 0x7FFFFFFFu) == 0x7F800000u;
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    const uint32_t u = __float_as_uint(v) & 0xFFFF0000u;
    o[k] = __ushort_as_bfloat16(static_cast<unsigned short>(u >> 16));
    v = inf ? 0.0f : v - __uint_as_float(u);
  }
}

}  // namespace

__global__ void __launch_bounds__(256) router_dz_kernel(const DzArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t t = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  if (t >= a.T) return;
  float dz[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) dz[i] = 0.0f;
  if (a.off) {
    const int s = seq_of(a.off, a.n_seq, t);
    if (s < a.n_seq && a.off[s] <= t) {
      const float L = static_cast<float>(static_cast<int64_t>(a.off[s + 1]) - a.off[s]);
      const float fl = static_cast<float>(a.Nr) / (static_cast<float>(a.Kr) * L);
      const float kk = (a.dloss ? a.dloss[s] : 1.0f) * (a.alpha / L);
      float v[EPL], f[EPL], om[EPL];
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const int e = lane + 32 * i;
        v[i] = f[i] = om[i] = 0.0f;
        if (e < a.Nr) {
          affinity_pair(a.partial, a.n_ks, a.T, a.Nr, t, e, v[i], om[i]);
          f[i] = fl * static_cast<float>(a.counts[static_cast<int64_t>(s) * a.Nr + e]);
        }
        sum += v[i];
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
      float fp = 0.0f;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        v[i] *= inv;
        fp = fmaf(f[i], v[i], fp);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) fp += __shfl_xor_sync(0xffffffffu, fp, o);
#pragma unroll
      for (int i = 0; i < EPL; ++i) dz[i] = kk * (v[i] * om[i]) * (f[i] - fp);
    }
  }
  if (a.dgate || a.gdot) {
    // lane r holds slot r
    int e = -1;
    float s = 0.0f, om = 0.0f;
    if (lane < a.Kr) {
      e = a.idx[t * a.Kr + lane];
      if (e < 0 || e >= a.Nr) {
        atomicOr(a.err, MOE_DEVERR_BAD_INDEX);
        e = -1;
      }
    }
    if (e >= 0) affinity_pair(a.partial, a.n_ks, a.T, a.Nr, t, e, s, om);
    float sum = s;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float gh = sum > 0.0f ? s / sum : 0.0f;
    float w = 0.0f;  // a_k
    if (e >= 0) {
      if (a.gdot) {
        const float *d = a.gdot + static_cast<int64_t>(a.pos[t * a.Kr + lane]) * a.n_dot;
        for (int j = 0; j < a.n_dot; ++j) w += d[j];
      } else {
        w = a.route_scale * a.dgate[t * a.Kr + lane] * gh;
      }
    }
    float tot = w;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) tot += __shfl_xor_sync(0xffffffffu, tot, o);
    const float d = om * (w - gh * tot);
    for (int r = 0; r < a.Kr; ++r) {
      const int er = __shfl_sync(0xffffffffu, e, r);
      const float dr = __shfl_sync(0xffffffffu, d, r);
      if (er >= 0 && (er & 31) == lane) {
#pragma unroll
        for (int i = 0; i < EPL; ++i)
          if (i == (er >> 5)) dz[i] += dr;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 32 * i;
    if (a.dlogits && e < a.Nr) a.dlogits[t * a.Nr + e] = dz[i];
    if (a.parts && e < a.Np) {
      __nv_bfloat16 o[3];
      split3(e < a.Nr ? dz[i] : 0.0f, o);
#pragma unroll
      for (int k = 0; k < 3; ++k) a.parts[(static_cast<int64_t>(k) * a.T + t) * a.Np + e] = o[k];
    }
  }
}

// --------------------------------------------------------------- dx = dz W_r
namespace {
constexpr int kParts = 3;
constexpr int RB_THREADS = 192;  // warp 0 TMA, warp 1 MMA, warps 2..5 epilogue
constexpr int RB_BOX = 128 * 128;  // one 32-column FP32 box of 128 rows
constexpr int X_STAGES = 4;
constexpr int X_A = 128 * 128;       // 128 tokens x 64 experts
constexpr int X_BG = 64 * 128;       // 64 experts x 64 columns
constexpr int X_B = 4 * 4 * X_BG;    // Np <= 256 experts x 256 columns
constexpr int X_SMEM = 1024 + X_B + X_STAGES * X_A + 2 * RB_BOX + 256;
static_assert(X_SMEM <= 232448, "shared memory budget");

struct DxArgs {
  int64_t T;
  int n_tiles, m_tiles, cols;  // 256-column strips, 128-token tiles, H
  int kb;                      // Np / 64
  int accumulate;
  int32_t *err;
  uint64_t limit_ns;
};

// 128 rows x 32 columns of FP32 per call: this thread's row `r` of the box.
__device__ __forceinline__ void put_box_row(uint8_t *box, int r, const uint32_t (&v)[32]) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    *reinterpret_cast<uint4 *>(box + r * 128 + ((j ^ (r & 7)) << 4)) =
        make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
}
}  // namespace

__global__ void __launch_bounds__(RB_THREADS, 1)
    router_dx_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_w,
                     const __grid_constant__ CUtensorMap map_o, const DxArgs args) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *sb = smem, *sa = smem + X_B, *so = sa + X_STAGES * X_A;
  uint64_t *full = reinterpret_cast<uint64_t *>(so + 2 * RB_BOX);
  uint64_t *empty = full + X_STAGES;
  uint64_t *bfull = empty + X_STAGES;
  uint64_t *tfull = bfull + 1;
  uint64_t *tempty = tfull + 2;
  uint64_t *teardown = tempty + 2;
  uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(teardown + 1);
  int *abort_flag = reinterpret_cast<int *>(tmem_holder + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < X_STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(bfull, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], 4);
    }
    mbar_init(teardown, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const WaitCtl ctl{abort_flag, args.err, args.limit_ns};
  const int nt = blockIdx.x % args.n_tiles, j0 = blockIdx.x / args.n_tiles;
  const int jn = gridDim.x / args.n_tiles;
  const int kb = args.kb, nk = kParts * kb;

  if (warp == 0) {
    if (lane == 0) {
      mbar_arrive_expect_tx(bfull, kb * 4 * X_BG);
      for (int b = 0; b < kb; ++b)
        for (int g = 0; g < 4; ++g)
          tma_load_2d(sb + (b * 4 + g) * X_BG, &map_w, bfull, nt * 256 + g * 64, b * 64);
      uint32_t it = 0;
      for (int m = j0; m < args.m_tiles && !*abort_flag; m += jn) {
        for (int k = 0; k < nk; ++k, ++it) {
          const int s = it % X_STAGES;
          if (!mbar_wait(&empty[s], ((it / X_STAGES) & 1) ^ 1, ctl)) break;
          mbar_arrive_expect_tx(&full[s], X_A);
          tma_load_2d(sa + s * X_A, &map_a, &full[s], (k % kb) * 64,
                      static_cast<int>((k / kb) * args.T + static_cast<int64_t>(m) * 128));
        }
      }
      // copies still in flight land before the CTA can exit
      int quiet = 0;
      const WaitCtl drain{&quiet, nullptr, 100000000ull};
      mbar_wait(bfull, 0, drain);
      const uint32_t n_inflight = it < X_STAGES ? it : X_STAGES;
      for (uint32_t q = it - n_inflight; q < it; ++q) mbar_wait(&full[q % X_STAGES], (q / X_STAGES) & 1, drain);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      uint32_t it = 0, tc = 0;
      const uint32_t idesc = idesc_bf16_f32(128, 256) | kIdescBMn;
      if (mbar_wait(bfull, 0, ctl)) {
        for (int m = j0; m < args.m_tiles && !*abort_flag; m += jn, ++tc) {
          const uint32_t buf = tc & 1;
          if (!mbar_wait(&tempty[buf], ((tc >> 1) & 1) ^ 1, ctl)) break;
          tc_fence_after();
          const uint32_t d = tmem + buf * 256;
          for (int k = 0; k < nk; ++k, ++it) {
            const int s = it % X_STAGES;
            if (!mbar_wait(&full[s], (it / X_STAGES) & 1, ctl)) break;
            tc_fence_after();
            const uint64_t da = sw128_kmajor_desc(smem_u32(sa + s * X_A));
            const uint64_t db = sw128_mnmajor_desc(smem_u32(sb + (k % kb) * 4 * X_BG), X_BG);
#pragma unroll
            for (int q = 0; q < 4; ++q)
              umma_bf16(d, da + 2 * q, db + (2048 >> 4) * q, idesc, (k > 0 || q > 0) ? 1u : 0u);
            umma_commit(&empty[s]);
          }
          umma_commit(&tfull[buf]);
        }
      }
      int quiet = 0;
      const WaitCtl drain{&quiet, nullptr, 100000000ull};
      umma_commit(teardown);
      mbar_wait(teardown, 0, drain);
    }
  } else {
    const int q = warp & 3;  // TMEM lane quarter
    const int r = q * 32 + lane;
    const bool issuer = warp == 2 && lane == 0;
    uint32_t tc = 0, nbox = 0;
    for (int m = j0; m < args.m_tiles; m += jn, ++tc) {
      const uint32_t buf = tc & 1;
      const bool ok = mbar_wait(&tfull[buf], (tc >> 1) & 1, ctl);
      // all four warps leave together (they meet at a barrier below)
      if (named_bar_or(1, 128, !ok)) break;
      tc_fence_after();
      const uint32_t ta = tmem + (static_cast<uint32_t>(q * 32) << 16) + buf * 256;
#pragma unroll 1
      for (int c = 0; c < 8; ++c) {
        const int x = nt * 256 + c * 32;
        if (x >= args.cols) break;
        uint32_t v[32];
        tmem_ld32(ta + c * 32, v);
        tmem_ld_wait();
        uint8_t *box = so + (nbox & 1) * RB_BOX;
        if (issuer) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
        named_bar_sync(1, 128);
        put_box_row(box, r, v);
        fence_proxy_async_smem();
        named_bar_sync(1, 128);
        if (issuer) {
          if (args.accumulate)
            tma_reduce_add_2d(&map_o, box, x, m * 128);
          else
            tma_store_2d(&map_o, box, x, m * 128);
          bulk_commit();
        }
        ++nbox;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty[buf]);
    }
    if (issuer) bulk_wait_all();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------ dW_r = dz^T x
namespace {
constexpr int WR_STAGES = 3;
constexpr int WR_TOK = 32;                       // tokens (K) per stage
constexpr int WR_G = WR_TOK * 128;               // 32 tokens x 64 experts (or columns)
constexpr int WR_A = kParts * 4 * WR_G;
constexpr int WR_B = 4 * WR_G;
constexpr int WR_STAGE = WR_A + WR_B;
constexpr int WR_SMEM = 1024 + WR_STAGES * WR_STAGE + 2 * RB_BOX + 256;
static_assert(WR_SMEM <= 232448, "shared memory budget");

struct DwrArgs {
  int64_t T;
  int n_tiles, n_split, cols;  // 256-column strips, token ranges, H
  int ng;                      // Np / 64
  int halves;                  // 128-expert halves
  int out_rows;                // output rows per token range
  int32_t *err;
  uint64_t limit_ns;
};
}  // namespace

__global__ void __launch_bounds__(RB_THREADS, 1)
    router_dwr_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_x,
                      const __grid_constant__ CUtensorMap map_o, const DwrArgs args) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *so = smem + WR_STAGES * WR_STAGE;
  uint64_t *full = reinterpret_cast<uint64_t *>(so + 2 * RB_BOX);
  uint64_t *empty = full + WR_STAGES;
  uint64_t *tfull = empty + WR_STAGES;
  uint64_t *teardown = tfull + 1;
  uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(teardown + 1);
  int *abort_flag = reinterpret_cast<int *>(tmem_holder + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < WR_STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(tfull, 1);
    mbar_init(teardown, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const WaitCtl ctl{abort_flag, args.err, args.limit_ns};
  const int nt = blockIdx.x % args.n_tiles, js = blockIdx.x / args.n_tiles;
  const int64_t nkb = (args.T + WR_TOK - 1) / WR_TOK;
  const int kb0 = static_cast<int>(js * nkb / args.n_split), kb1 = static_cast<int>((js + 1) * nkb / args.n_split);

  if (warp == 0) {
    if (lane == 0) {
      uint32_t it = 0;
      for (int kb = kb0; kb < kb1; ++kb, ++it) {
        const int s = it % WR_STAGES;
        if (!mbar_wait(&empty[s], ((it / WR_STAGES) & 1) ^ 1, ctl)) break;
        uint8_t *st = smem + s * WR_STAGE;
        mbar_arrive_expect_tx(&full[s], (kParts * args.ng + 4) * WR_G);
        for (int g = 0; g < 4; ++g)
          tma_load_2d(st + WR_A + g * WR_G, &map_x, &full[s], nt * 256 + g * 64, kb * WR_TOK);
        for (int p = 0; p < kParts; ++p)
          for (int g = 0; g < args.ng; ++g)
            tma_load_2d(st + (p * 4 + g) * WR_G, &map_a, &full[s], g * 64,
                        static_cast<int>(p * args.T + static_cast<int64_t>(kb) * WR_TOK));
      }
      int quiet = 0;
      const WaitCtl drain{&quiet, nullptr, 100000000ull};
      const uint32_t n_inflight = it < WR_STAGES ? it : WR_STAGES;
      for (uint32_t q = it - n_inflight; q < it; ++q) mbar_wait(&full[q % WR_STAGES], (q / WR_STAGES) & 1, drain);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      uint32_t it = 0;
      const uint32_t idesc = idesc_bf16_f32(128, 256) | kIdescAMn | kIdescBMn;
      for (int kb = kb0; kb < kb1; ++kb, ++it) {
        const int s = it % WR_STAGES;
        if (!mbar_wait(&full[s], (it / WR_STAGES) & 1, ctl)) break;
        tc_fence_after();
        const uint32_t st = smem_u32(smem + s * WR_STAGE);
#pragma unroll
        for (int q = 0; q < WR_TOK / 16; ++q) {
          const uint64_t db = sw128_mnmajor_desc(st + WR_A + q * 2048, WR_G);
#pragma unroll
          for (int p = 0; p < kParts; ++p)
            for (int h = 0; h < args.halves; ++h)
              umma_bf16(tmem + h * 256, sw128_mnmajor_desc(st + (p * 4 + h * 2) * WR_G + q * 2048, WR_G), db, idesc,
                        (it > 0 || q > 0 || p > 0) ? 1u : 0u);
        }
        umma_commit(&empty[s]);
      }
      umma_commit(tfull);
      int quiet = 0;
      const WaitCtl drain{&quiet, nullptr, 100000000ull};
      umma_commit(teardown);
      mbar_wait(teardown, 0, drain);
    }
  } else {
    const int q = warp & 3;
    const int r = q * 32 + lane;
    const bool issuer = warp == 2 && lane == 0;
    const bool ok = mbar_wait(tfull, 0, ctl);
    if (!named_bar_or(1, 128, !ok)) {
      tc_fence_after();
      uint32_t nbox = 0;
      for (int h = 0; h < args.halves; ++h) {
        const uint32_t ta = tmem + (static_cast<uint32_t>(q * 32) << 16) + h * 256;
#pragma unroll 1
        for (int c = 0; c < 8; ++c) {
          const int x = nt * 256 + c * 32;
          if (x >= args.cols) break;
          uint32_t v[32];
          tmem_ld32(ta + c * 32, v);
          tmem_ld_wait();
          uint8_t *box = so + (nbox & 1) * RB_BOX;
          if (issuer) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
          named_bar_sync(1, 128);
          put_box_row(box, r, v);
          fence_proxy_async_smem();
          named_bar_sync(1, 128);
          if (issuer) {
            tma_store_2d(&map_o, box, x, js * args.out_rows + h * 128);
            bulk_commit();
          }
          ++nbox;
        }
      }
      tc_fence_before();
    }
    if (issuer) bulk_wait_all();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// part [n, rows, cols] -> out [Nr, cols], the ranges in order; 4 columns a thread
__global__ void __launch_bounds__(256) dwr_join_kernel(const float *__restrict__ part, int n, int rows, int Nr,
                                                        int cols, float *__restrict__ out) {
  const int64_t i = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) * 4;
  if (i >= static_cast<int64_t>(Nr) * cols) return;
  const int64_t stride = static_cast<int64_t>(rows) * cols;
  float4 s = *reinterpret_cast<const float4 *>(part + i);
  for (int k = 1; k < n; ++k) {
    const float4 v = *reinterpret_cast<const float4 *>(part + k * stride + i);
    s.x += v.x;
    s.y += v.y;
    s.z += v.z;
    s.w += v.w;
  }
  *reinterpret_cast<float4 *>(out + i) = s;
}

// -------------------------------------------------------------------- host
int router_parts_pitch(int Nr) { return (Nr + 63) / 64 * 64; }

// Token ranges of the dW_r product: as many as fill the SMs in one wave.
int router_dwr_split(int64_t T, int cols) {
  const int n_tiles = (cols + 255) / 256;
  const int64_t nkb = (T + WR_TOK - 1) / WR_TOK;
  int64_t j = moe_host::sm_count() / n_tiles;
  if (j > nkb) j = nkb;
  return static_cast<int>(j < 1 ? 1 : j);
}
int router_dwr_rows(int Nr) { return (Nr + 127) / 128 * 128; }

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
  router_dz_kernel<<<static_cast<unsigned>((g.T + 7) / 8), 256, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_router_dx(const void *parts, const void *wr, int64_t T, int Nr, int H, float *dx, int accumulate,
                             int32_t *err, uint64_t limit_ns, cudaStream_t st) {
  if (T == 0) return cudaSuccess;
  const int Np = router_parts_pitch(Nr);
  CUtensorMap ma, mw, mo;
  if (moe_host::encode_tmap_2d(&ma, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, parts, Np, kParts * T,
                               static_cast<uint64_t>(Np) * 2, 64, 128) != 0 ||
      moe_host::encode_tmap_2d(&mw, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, wr, H, Nr, static_cast<uint64_t>(H) * 2, 64,
                               64) != 0 ||
      moe_host::encode_tmap_2d(&mo, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, dx, H, T, static_cast<uint64_t>(H) * 4, 32,
                               128) != 0)
    return cudaErrorInvalidValue;
  DxArgs a{};
  a.T = T;
  a.cols = H;
  a.n_tiles = (H + 255) / 256;
  a.m_tiles = static_cast<int>((T + 127) / 128);
  a.kb = Np / 64;
  a.accumulate = accumulate;
  a.err = err;
  a.limit_ns = limit_ns;
  static std::atomic<uint64_t> attr_done{0};
  if (const cudaError_t e = smem_attr_once(router_dx_kernel, X_SMEM, attr_done)) return e;
  int j = moe_host::sm_count() / a.n_tiles;
  if (j > a.m_tiles) j = a.m_tiles;
  if (j < 1) j = 1;
  router_dx_kernel<<<a.n_tiles * j, RB_THREADS, X_SMEM, st>>>(ma, mw, mo, a);
  return cudaGetLastError();
}

cudaError_t launch_router_dwr(const void *parts, const void *x, int64_t T, int Nr, int H, float *part, float *dwr,
                              int32_t *err, uint64_t limit_ns, cudaStream_t st) {
  if (T == 0) return cudaMemsetAsync(dwr, 0, sizeof(float) * Nr * static_cast<size_t>(H), st);
  const int Np = router_parts_pitch(Nr);
  DwrArgs a{};
  a.T = T;
  a.cols = H;
  a.n_tiles = (H + 255) / 256;
  a.n_split = router_dwr_split(T, H);
  a.ng = Np / 64;
  a.halves = (Nr + 127) / 128;
  a.out_rows = router_dwr_rows(Nr);
  a.err = err;
  a.limit_ns = limit_ns;
  const bool join = a.n_split > 1;
  CUtensorMap ma, mx, mo;
  if (moe_host::encode_tmap_2d(&ma, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, parts, Np, kParts * T,
                               static_cast<uint64_t>(Np) * 2, 64, WR_TOK) != 0 ||
      moe_host::encode_tmap_2d(&mx, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, x, H, T, static_cast<uint64_t>(H) * 2, 64,
                               WR_TOK) != 0 ||
      moe_host::encode_tmap_2d(&mo, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, join ? part : dwr, H,
                               join ? static_cast<uint64_t>(a.n_split) * a.out_rows : Nr,
                               static_cast<uint64_t>(H) * 4, 32, 128) != 0)
    return cudaErrorInvalidValue;
  static std::atomic<uint64_t> attr_done{0};
  if (const cudaError_t e = smem_attr_once(router_dwr_kernel, WR_SMEM, attr_done)) return e;
  router_dwr_kernel<<<a.n_tiles * a.n_split, RB_THREADS, WR_SMEM, st>>>(ma, mx, mo, a);
  if (const cudaError_t e = cudaGetLastError()) return e;
  if (join) {
    const int64_t n4 = static_cast<int64_t>(Nr) * H / 4;
    dwr_join_kernel<<<static_cast<unsigned>((n4 + 255) / 256), 256, 0, st>>>(part, a.n_split, a.out_rows, Nr, H, dwr);
  }
  return cudaGetLastError();
}

}  // namespace moe
