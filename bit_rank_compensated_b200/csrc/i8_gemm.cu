// The 8-bit linear's product: Y[m, n] = (sum_k xq[m, k] wq[n, k]) x_scale[m] w_scale[n] + bias[n], with
// exact 32-bit integer sums.
//
// Persistent kernel of CTA pairs (clusters of two CTAs on two SMs). A pair owns an output tile of
// 256 tokens x 256 channels and computes it with cta_group::2 kind::i8 tensor-core MMAs of M = N = 256,
// K = 32: each CTA stages its own 128 rows of xq and its own 128 rows of wq, 128 columns of K per
// pipeline step (128-byte rows, 128B swizzle), the even CTA issues the MMAs for both, and each CTA's
// tensor memory holds the sums of its 128 tokens. Two accumulators (all 512 tensor-memory columns) let
// the output stage drain one tile while the next one's MMAs run.
//
// The scales multiply the sum once per element, in the output stage: the integer part of the
// product needs no scale, so int8 runs with no scale traffic in the loop (the 4-bit GEMM's blocks).
//
// What was measured: a step takes 0.28 us (550 cycles, 512 of them the MMAs') while the chip is not
// full. There is one tile: for 16 tokens, 4096 x 4096, narrower ones took as long (256, 192, 128 and 64 channels:
// 13.4, 12.9, 12.8 and 13.4 us, with an earlier output stage), since the weights' way in bounds them there. Where
// the last wave of tiles is nearly empty (2202 x 4608: 162 tiles on 74 pairs take three waves for 2.2) a narrower
// one was not measured. Four output groups instead of two cost 1.5 us a launch and 3 % of the large product. The output stage takes 2850 cycles a
// tile (4100 to 6200 with a row to a thread, which reads every scale; converting the sums by
// integer arithmetic instead of the conversion instruction made it slower).
// Where there are at most half as many tiles as pairs, the K axis is split: each pair writes the raw sums of
// its share and a second kernel adds them (integers: in any order the same) and applies the scales.
//
// Warp roles (384 threads): warp 0 TMA producer; warp 1 tensor-memory owner and, in the even CTA, MMA
// issuer; warps 2, 3 idle; warps 4..11 output stage, two groups of four warps, each 128 of the tile's
// columns. An output thread scales its share of 16 x 8 blocks, rounds once and writes to one of two swizzled
// boxes, in turn, which TMA stores clip to M and N. Every wait is bounded.
#include <type_traits>

#include "block.h"
#include "common.cuh"
#include "types.cuh"

namespace svdq {
namespace {

constexpr int BM = 128;  // tokens per CTA, 256 per pair
constexpr int STEP = 128;  // columns of K per pipeline step
constexpr int BN = 256;  // channels per pair
constexpr int EPI_WARP0 = 4;
constexpr int GROUPS = 2;  // output groups of four warps
constexpr int COLS = BN / GROUPS;  // columns of a group
constexpr int THREADS = 32 * EPI_WARP0 + 128 * GROUPS;
constexpr int ST = 5;  // stages
constexpr int BOXES = 2;  // output boxes of a group
constexpr uint32_t A_BYTES = BM * STEP;
constexpr uint32_t B_BYTES = BN / 2 * STEP;
constexpr uint32_t STAGE_BYTES = A_BYTES + B_BYTES;
constexpr uint32_t BOX_BYTES = BM * 128;  // output box: 128 rows of 128 bytes
constexpr uint32_t DATA_BYTES = ST * STAGE_BYTES;
constexpr int N_BARS = 2 * ST + 4;
constexpr uint32_t SMEM = DATA_BYTES + GROUPS * BOXES * BOX_BYTES + 256 + 1024;
constexpr uint32_t TMEM_COLS = 512;
static_assert(SMEM <= 232448, "shared memory per CTA");
static_assert(N_BARS * 8 + 4 <= 256, "barrier area");
static_assert(STAGE_BYTES % 1024 == 0, "stages keep the 1 KiB alignment of 128B-swizzled tiles");
static_assert(2 * BN <= TMEM_COLS, "two accumulators");

struct GArgs {
  const float *x_scale, *w_scale, *bias;
  int M, N, K;
  int Mt, Nt;
  int splits, split_steps;  // shares of the K axis and the steps of each
  uint32_t *err;
};

// A value from its sum: scaled in fp32, one fp32 rounding each for the sum, the two scales and the bias.
__device__ __forceinline__ float scaled(int acc, float xs, float ws, float b) {
  return fmaf(__fmul_rn(static_cast<float>(acc), xs), ws, b);
}

// T: type of Y, or int for the raw sums of a share of the K axis (tm_y then has M x N for each share).
template <typename T>
__global__ void __launch_bounds__(THREADS, 1) __cluster_dims__(2, 1, 1)
    k_i8_gemm(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
              const __grid_constant__ CUtensorMap tm_y, GArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *box_s = smem + DATA_BYTES;
  uint64_t *bars = reinterpret_cast<uint64_t *>(box_s + GROUPS * BOXES * BOX_BYTES);
  // full[s] (even CTA): stage s is loaded in both CTAs; empty[s]: the MMAs that read it are done (both
  // CTAs); accfull[b]: accumulator b is complete (both CTAs); accempty[b] (even CTA): both CTAs have read it
  const uint32_t bar_full = smem_u32(bars), bar_empty = bar_full + 8 * ST;
  const uint32_t bar_accfull = bar_empty + 8 * ST, bar_accempty = bar_accfull + 16;
  uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(bars + N_BARS);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t crank = cluster_ctarank();
  const int pid = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  const int steps = (a.K + STEP - 1) / STEP;
  const int mn = a.Mt * a.Nt;
  const int tiles = mn * a.splits;  // tile t: output tile t % mn, share t / mn

  if (threadIdx.x == 0) {
    for (int s = 0; s < ST; ++s) {
      mbar_init(bar_full + 8 * s, 1);
      mbar_init(bar_empty + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar_accfull + 8 * b, 1);
      mbar_init(bar_accempty + 8 * b, 2 * 4 * GROUPS);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_holder), TMEM_COLS);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tbase = *tmem_holder;
  // global memory only from here on: the prologue overlaps the previous kernel of the stream
  grid_dep_wait();
  grid_dep_launch();

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      tma_prefetch_desc(&tm_x);
      tma_prefetch_desc(&tm_w);
      uint32_t it = 0;
      bool ok = true;
      for (int t = pid; t < tiles && ok; t += npairs) {
        const int o = t % mn, j0 = t / mn * a.split_steps;
        const int row0 = (o % a.Mt) * 2 * BM + static_cast<int>(crank) * BM;
        const int wrow0 = (o / a.Mt) * BN + static_cast<int>(crank) * (BN / 2);
        const int j1 = min(steps, j0 + a.split_steps);
        for (int j = j0; j < j1; ++j, ++it) {
          const int s = it % ST;
          if (it >= ST && !mbar_wait_parked(bar_empty + 8 * s, ((it / ST) - 1) & 1, a.err, KID_I8, 1)) {
            ok = false;
            break;
          }
          const uint32_t lead = map_shared_rank(bar_full + 8 * s, 0);
          const uint32_t at = smem_u32(smem + s * STAGE_BYTES);
          if (crank == 0) mbar_arrive_expect_tx(bar_full + 8 * s, 2 * STAGE_BYTES);
          tma_load_2d_pair(at, &tm_x, j * STEP, row0, lead);
          tma_load_2d_pair(at + A_BYTES, &tm_w, j * STEP, wrow0, lead);
        }
      }
      // the MMA issuer's last commits to this CTA's barriers have landed before it exits
      for (uint32_t i = it > ST ? it - ST : 0; ok && i < it; ++i)
        ok = mbar_wait(bar_empty + 8 * (i % ST), (i / ST) & 1, a.err, KID_I8, 2);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (even CTA)
    if (crank == 0) {
      // kind::i8: D int32 (bits 4-5 = 2), A and B int8 (bits 7-9, 10-12 = 1), K-major, N (bits 17-22),
      // M = 256 across the pair (bits 24-28)
      constexpr uint32_t idesc = (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t(BN) >> 3) << 17) | ((256u >> 4) << 24);
      uint32_t it = 0, n = 0;
      bool ok = true;
      for (int t = pid; t < tiles && ok; t += npairs, ++n) {
        const uint32_t b = n & 1;
        if (n >= 2 && !__all_sync(0xffffffffu, mbar_wait(bar_accempty + 8 * b, ((n >> 1) - 1) & 1, a.err, KID_I8, 3))) break;
        tc_fence_after();
        const int j0 = t / mn * a.split_steps, j1 = min(steps, j0 + a.split_steps);
        for (int j = j0; j < j1; ++j, ++it) {
          const int s = it % ST;
          if (!__all_sync(0xffffffffu, mbar_wait(bar_full + 8 * s, (it / ST) & 1, a.err, KID_I8, 4))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t at = smem_u32(smem + s * STAGE_BYTES);
          const uint64_t ad = umma_desc(at, 16, 1024, 2), bd = umma_desc(at + A_BYTES, 16, 1024, 2);
          const int kb = min(4, (a.K - j * STEP + 31) / 32);  // columns beyond K are zeros: whole MMAs of them are left out
          if (elect_one()) {
            for (int k = 0; k < kb; ++k)
              mma_i8_pair(tbase + b * BN, ad + 2u * k, bd + 2u * k, idesc, j > j0 || k > 0 ? 1u : 0u);
            tc_commit_pair_mc(bar_empty + 8 * s, 0x3);
          }
          __syncwarp();
        }
        if (!ok) break;
        if (elect_one()) tc_commit_pair_mc(bar_accfull + 8 * b, 0x3);
        __syncwarp();
      }
      // the output stages of both CTAs have released the last accumulators
      for (uint32_t i = n > 2 ? n - 2 : 0; ok && i < n; ++i)
        ok = __all_sync(0xffffffffu, mbar_wait(bar_accempty + 8 * (i & 1), (i >> 1) & 1, a.err, KID_I8, 5));
    }
  } else if (warp >= EPI_WARP0) {
    // ------------------------------------------------------------ output stage
    const int group = (warp - EPI_WARP0) >> 2, quad = warp & 3;
    const int et = (static_cast<int>(threadIdx.x) - EPI_WARP0 * 32) & 127;  // thread of the group
    // This thread's elements of a 16-row, 8-column block: rows lane / 4 and 8 further, columns 2 (lane % 4) and
    // the next (the 16x256b loads' layout). A thread so needs the scales of a quarter of the columns and of
    // four rows; with a row to a thread the scales' way from shared memory (every thread all of them) took
    // most of the output stage's time.
    const int row = quad * 32 + lane / 4, col = 2 * (lane % 4);
    const uint32_t tlane = static_cast<uint32_t>(quad * 32) << 16;
    constexpr bool RAW = std::is_same_v<T, int>;
    constexpr int PER_BOX = 128 / sizeof(T);  // columns of a box
    constexpr int BLOCKS = PER_BOX / 8;       // 8-column blocks of a box
    // shared addresses: the pointers' state space is lost in their alignment, and generic accesses are slower
    const uint32_t boxes = smem_u32(box_s + group * BOXES * BOX_BYTES);
    uint32_t turn = 0;  // boxes filled
    bool ok = true;
    uint32_t n = 0;
    for (int t = pid; t < tiles; t += npairs, ++n) {
      const uint32_t b = n & 1;
      const int o = t % mn;
      const int row0 = (o % a.Mt) * 2 * BM + static_cast<int>(crank) * BM;
      const int n0 = (o / a.Mt) * BN + group * COLS;
      // this thread's scales and bias, on their way while the MMAs run (N is even: a pair lies inside or outside)
      float xs[4] = {};
      float2 ws2[COLS / 8], bs2[COLS / 8];
      if constexpr (!RAW) {
#pragma unroll
        for (int i = 0; i < 4; ++i) xs[i] = row0 + row + 8 * i < a.M ? __ldg(a.x_scale + row0 + row + 8 * i) : 0.0f;
#pragma unroll
        for (int j = 0; j < COLS / 8; ++j) {
          const int nc = n0 + 8 * j + col;
          ws2[j] = nc < a.N ? make_float2(__ldg(a.w_scale + nc), __ldg(a.w_scale + nc + 1)) : make_float2(0.0f, 0.0f);
          bs2[j] = a.bias && nc < a.N ? make_float2(__ldg(a.bias + nc), __ldg(a.bias + nc + 1)) : make_float2(0.0f, 0.0f);
        }
      }
      if (ok) ok = mbar_wait_parked(bar_accfull + 8 * b, (n >> 1) & 1, a.err, KID_I8, 6);
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
      const uint32_t taddr = tbase + tlane + b * BN + group * COLS;
#pragma unroll
      for (int c = 0; c < COLS; c += PER_BOX) {
        // the box's words: scaled, rounded and packed before the box has to be free
        uint32_t w[2][2][BLOCKS][sizeof(T) / 2];  // [16 rows][8 rows][block][word]
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t r[4 * BLOCKS];
          if (ok) tmem_ld_16x256b(taddr + (static_cast<uint32_t>(16 * half) << 16) + c, r);
          if (half == 1 && c + PER_BOX == COLS) {
            // the sums are in registers: the accumulator goes back to the MMAs
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(map_shared_rank(bar_accempty + 8 * b, 0));
          }
#pragma unroll
          for (int j = 0; j < BLOCKS; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t r0 = r[4 * j + 2 * i], r1 = r[4 * j + 2 * i + 1];
              if constexpr (RAW) {
                w[half][i][j][0] = r0;
                w[half][i][j][1] = r1;
              } else {
                const float v0 = scaled(static_cast<int>(r0), xs[2 * half + i], ws2[c / 8 + j].x, bs2[c / 8 + j].x);
                const float v1 = scaled(static_cast<int>(r1), xs[2 * half + i], ws2[c / 8 + j].y, bs2[c / 8 + j].y);
                if constexpr (sizeof(T) == 4) {
                  w[half][i][j][0] = __float_as_uint(v0);
                  w[half][i][j][1] = __float_as_uint(v1);
                } else {
                  w[half][i][j][0] = narrow(pair(v0, v1), T{});
                }
              }
            }
        }
        // the box is free once the copy unit has read what it held two boxes ago
        if (et == 0) bulk_wait_read1();
        named_bar_sync(1 + group, 128);
        const uint32_t box = boxes + (turn++ & 1 ? BOX_BYTES : 0u);
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int rw = row + 16 * half + 8 * i;
            const uint32_t at = box + rw * 128;
#pragma unroll
            for (int j = 0; j < BLOCKS; ++j) {
              // 16-byte chunk k of a row lies at k ^ (row % 8)
              if constexpr (sizeof(T) == 4) {
                const int k = 2 * j + (lane % 4) / 2;
                st_shared_u32x2(at + ((k ^ (rw & 7)) << 4) + 8 * (lane % 2), w[half][i][j][0], w[half][i][j][1]);
              } else {
                st_shared_u32(at + ((j ^ (rw & 7)) << 4) + 4 * (lane % 4), w[half][i][j][0]);
              }
            }
          }
        fence_proxy_async_smem();
        named_bar_sync(1 + group, 128);
        if (et == 0) {
          if (ok && n0 + c < a.N && row0 < a.M) {
            if constexpr (RAW) tma_store_3d(&tm_y, box, n0 + c, row0, t / mn);
            else tma_store_2d(&tm_y, box, n0 + c, row0);
          }
          bulk_commit();
        }
      }
    }
    if (et == 0) bulk_wait0();  // stores complete before the CTA exits
  }

  __syncthreads();
  tc_fence_before();
  cluster_sync_all();  // neither CTA frees the pair's tensor memory while the other still uses it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tbase, TMEM_COLS);
  }
}

// Y from the sums of the K axis's shares: four channels a thread.
template <typename T>
__global__ void __launch_bounds__(256) k_i8_shares(const int *part, GArgs a, T *Y) {
  grid_dep_wait();
  grid_dep_launch();
  const size_t size = static_cast<size_t>(a.M) * a.N;
  const size_t i = 4 * (static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x);
  if (i >= size) return;
  const int m = static_cast<int>(i / a.N), n = static_cast<int>(i % a.N);
  int4 s = make_int4(0, 0, 0, 0);
#pragma unroll 4
  for (int j = 0; j < a.splits; ++j) {
    const int4 v = *reinterpret_cast<const int4 *>(part + j * size + i);
    s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
  }
  const float xs = a.x_scale[m];
  const float ws[4] = {a.w_scale[n], a.w_scale[n + 1], a.w_scale[n + 2], a.w_scale[n + 3]};
  float b[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (a.bias)
#pragma unroll
    for (int e = 0; e < 4; ++e) b[e] = a.bias[n + e];
  const float v[4] = {scaled(s.x, xs, ws[0], b[0]), scaled(s.y, xs, ws[1], b[1]), scaled(s.z, xs, ws[2], b[2]), scaled(s.w, xs, ws[3], b[3])};
  if constexpr (sizeof(T) == 4) *reinterpret_cast<float4 *>(Y + i) = make_float4(v[0], v[1], v[2], v[3]);
  else *reinterpret_cast<uint2 *>(Y + i) = make_uint2(narrow(pair(v[0], v[1]), T{}), narrow(pair(v[2], v[3]), T{}));
}

int steps_of(int K) { return (K + STEP - 1) / STEP; }

// Shares of the K axis. A pair's steps take 0.28 us each, and what a split adds is the second kernel
// (about 2 us) and the shares' way through L2 (4 bytes written and read for each share and element, at
// about 5 TB/s): split into the number of shares for which the sum is least,
// of four steps at least and no more than there are pairs to take them.
int splits_of(int M, int N, int K, int pairs) {
  const int64_t tiles = static_cast<int64_t>(pieces(M, 2 * BM)) * pieces(N, BN);
  const int steps = steps_of(K);
  if (2 * tiles > pairs) return 1;
  int most = static_cast<int>(pairs / tiles);
  if (most > steps / 4) most = steps / 4;
  if (most > 16) most = 16;
  int best = 1;
  double least = 0.28 * steps;
  for (int s = 2; s <= most; ++s) {
    const int each = (steps + s - 1) / s;
    if ((steps + each - 1) / each != s) continue;  // s shares would leave some empty
    const double t = 0.28 * each + 2.0 + 8.0 * s * static_cast<double>(M) * N / 5e6;
    if (t < least) {
      least = t;
      best = s;
    }
  }
  return best;
}
constexpr int kPairs = 74;  // SM pairs of a B200: the split, and so the workspace, depends on sizes alone

template <typename T>
cudaError_t launch_t(const I8GemmLaunch &g) {
  const int splits = splits_of(g.M, g.N, g.K, kPairs);
  const int each = (steps_of(g.K) + splits - 1) / splits;
  CUtensorMap tx, tw, ty;
  const uint64_t K = g.K, e = sizeof(T);
  constexpr CUtensorMapDataType dt = sizeof(T) == 4              ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                     : std::is_same_v<T, __half> ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                                 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  if (!make_map(&tx, CU_TENSOR_MAP_DATA_TYPE_UINT8, g.xq, K, g.M, K, STEP, BM, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_map(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, g.wq, K, g.N, K, STEP, BN / 2, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  const bool mapped = splits > 1 ? make_map_3d(&ty, CU_TENSOR_MAP_DATA_TYPE_INT32, g.workspace, g.N, g.M, splits, 4, 32, BM, CU_TENSOR_MAP_SWIZZLE_128B)
                                 : make_map(&ty, dt, g.Y, g.N, g.M, g.N * e, 128 / e, BM, CU_TENSOR_MAP_SWIZZLE_128B);
  if (!mapped) return cudaErrorInvalidValue;
  const GArgs a{g.x_scale, g.w_scale, g.bias, g.M, g.N, g.K, pieces(g.M, 2 * BM), pieces(g.N, BN), splits, each, g.dev->err};
  auto kern = splits > 1 ? k_i8_gemm<int> : k_i8_gemm<T>;
  cudaError_t err = allow_smem<SMEM>(kern);
  if (err != cudaSuccess) return err;
  const int64_t tiles = static_cast<int64_t>(a.Mt) * a.Nt * splits;
  const int slots = g.dev->num_sms / 2;
  const dim3 grid(2 * static_cast<unsigned>(tiles < slots ? tiles : slots));
  err = launch_dependent(kern, grid, THREADS, SMEM, g.stream, tx, tw, ty, a);
  if (err != cudaSuccess || splits == 1) return err;
  const size_t quads = static_cast<size_t>(g.M) * g.N / 4;
  return launch_dependent(k_i8_shares<T>, dim3(static_cast<unsigned>((quads + 255) / 256)), 256, 0, g.stream,
                          static_cast<const int *>(g.workspace), a, static_cast<T *>(g.Y));
}

}  // namespace

size_t i8_gemm_workspace_bytes(int M, int N, int K) {
  if (i8_few_fits(M, N, K)) return 0;
  const int s = splits_of(M, N, K, kPairs);
  return s > 1 ? 4 * static_cast<size_t>(s) * M * N : 0;
}

cudaError_t launch_i8_gemm(const I8GemmLaunch &g) {
  if (i8_few_fits(g.M, g.N, g.K)) return launch_i8_few(g);
  if (static_cast<int64_t>(pieces(g.M, 2 * BM)) * pieces(g.N, BN) >= (1ll << 30)) return cudaErrorInvalidValue;
  if (g.y_dtype == SVDQ_F32) return launch_t<float>(g);
  if (g.y_dtype == SVDQ_F16) return launch_t<__half>(g);
  return launch_t<__nv_bfloat16>(g);
}

}  // namespace svdq
