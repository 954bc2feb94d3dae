// linear.cuh - dense matrix product with a fused epilogue on tcgen05.
//
//   y[t, n] = round( act( x_scale[t] * w_scale[n] * sum_k x[t, k] w[n, k] + bias[n] ) + residual[t, n] )
//
// x [T, K] and w [N, K] are read by TMA in 128-byte K atoms (64 values of 16
// bits, 128 of 8; the tensor map zero-fills past K, T and N, so any T, N and K
// runs), the sum is kept in fp32 in TMEM, everything after it happens in
// registers, and the result is rounded once.
//
// k_linear_split: weights on the MMA's M side (128 outputs per tile), up to BN
// tokens on N, and the K axis split over the S CTAs of a cluster. Each CTA
// leaves its fp32 partial tile in its own shared memory; after a cluster
// barrier every CTA adds the S partials of its share of the token columns over
// distributed shared memory, in rank order, and finishes them. No workspace,
// no atomics: the result does not depend on the order in which CTAs finish.
// What bounds it: with few tokens the weights' stream from HBM, N * K * size
// bytes, which needs all SMs pulling at once; the K split is what supplies them
// when N / 128 tiles are fewer than the SMs.
#pragma once
#include "gemm.cuh"
#include "router.cuh"

namespace moe {

enum LinearAct : int { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4, kActSigmoid = 5 };

struct LinearArgs {
  int T, N;
  int nk;                // K atoms
  int f16;               // 16-bit operands are fp16
  const float* x_scale;  // [T] or nullptr (8-bit operands)
  const float* w_scale;  // [N], or one value with w_scale_step = 0
  int w_scale_step;
  const void* bias;  // [N] or nullptr
  int bias_dt;
  int act;
  const void* residual;  // rows ldr apart, in the output's type, or nullptr
  size_t ldr;
  void* out;  // rows ldo apart
  size_t ldo;
  int out_dt;  // MOE_DT_BF16, MOE_DT_FP16 or MOE_DT_F32
  int n_tb;    // token blocks
};

// Instruction descriptor of kind::f16 with both operands bf16 or both fp16.
__host__ __device__ constexpr uint32_t idesc_16bit(int M, int N, bool f16) {
  return f16 ? idesc_bf16(M, N) & ~((7u << 7) | (7u << 10)) : idesc_bf16(M, N);
}

// The activation of C accumulated values. The exponentials are the fast ones
// (relative error near 2^-21, far below a 16-bit output's rounding and of the
// size of the fp32 accumulation's own error). NaN passes through every one.
template <int C>
__device__ __forceinline__ void apply_act(float (&v)[C], int act) {
  switch (act) {
    case kActRelu:
#pragma unroll
      for (int i = 0; i < C; ++i) v[i] = v[i] < 0.f ? 0.f : v[i];
      break;
    case kActSilu:
#pragma unroll
      for (int i = 0; i < C; ++i) v[i] = __fdividef(v[i], 1.0f + __expf(-v[i]));
      break;
    case kActGelu:  // v * Phi(v), by the complementary error function: no cancellation in the left tail
#pragma unroll
      for (int i = 0; i < C; ++i) v[i] = 0.5f * v[i] * erfcf(-0.70710678118654752f * v[i]);
      break;
    case kActGeluTanh:  // 0.5 v (1 + tanh u) = v / (1 + exp(-2u))
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const float u2 = 1.5957691216057308f * (v[i] + 0.044715f * v[i] * v[i] * v[i]);
        v[i] = __fdividef(v[i], 1.0f + __expf(-u2));
      }
      break;
    case kActSigmoid:
#pragma unroll
      for (int i = 0; i < C; ++i) v[i] = __fdividef(1.0f, 1.0f + __expf(-v[i]));
      break;
    default: break;
  }
}

__device__ __forceinline__ float load_typed(const void* p, int dt, size_t i) {
  if (dt == 4) return __ldg(static_cast<const float*>(p) + i);
  const unsigned short b = __ldg(static_cast<const unsigned short*>(p) + i);
  return dt == 0 ? __bfloat162float(__ushort_as_bfloat16(b)) : __half2float(__ushort_as_half(b));
}

// The residual may be the output itself: no read-only load.
__device__ __forceinline__ float load_residual(const void* p, int dt, size_t i) {
  if (dt == 4) return static_cast<const float*>(p)[i];
  if (dt == 0) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  return __half2float(static_cast<const __half*>(p)[i]);
}

__device__ __forceinline__ void store_typed(void* p, int dt, size_t i, float v) {
  if (dt == 4) static_cast<float*>(p)[i] = v;
  else if (dt == 0) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else static_cast<__half*>(p)[i] = __float2half_rn(v);
}

__device__ __forceinline__ float ld_shared_cluster_f32(uint32_t cluster_addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr) : "memory");
  return v;
}

// ------------------------------------------------------------ K split over a cluster

constexpr int kSplitThreads = 192;  // producer, MMA, four epilogue warps

template <int BN>
struct SplitCfg {
  static constexpr int kStageBytes = (kTileM + BN) * kTileKBytes;
  // about 100 KB of operands in flight per CTA up to 64 tokens (two CTAs per
  // SM), all of shared memory above
  static constexpr int kStages = BN == 16 ? 5 : BN == 32 ? 5 : BN == 64 ? 4 : BN == 128 ? 6 : 4;
  static constexpr int kBarOffset = kStages * kStageBytes;
  static constexpr int kBytes = kBarOffset + (2 * kStages + 2) * 8 + 16 + 1024;  // + alignment slack
  static constexpr int kTmemCols = BN < 32 ? 32 : BN;
  static_assert(kStageBytes % 1024 == 0, "stages start on 1024-byte swizzle boundaries");
  static_assert(BN * kTileM * 4 <= kBarOffset, "the partial tile fits the stages it replaces");
};

// Scale, bias, activation, residual and store of C tokens t0.. of output n.
template <int C>
__device__ __forceinline__ void split_finish(const LinearArgs& g, float (&v)[C], int n, int t0, int t_end, float ws,
                                             float bias) {
  float r[C];
#pragma unroll
  for (int i = 0; i < C; ++i) r[i] = 0.f;
  if (g.residual) {
#pragma unroll
    for (int i = 0; i < C; ++i)
      if (t0 + i < t_end) r[i] = load_residual(g.residual, g.out_dt, (t0 + i) * g.ldr + n);
  }
  if (g.x_scale) {
#pragma unroll
    for (int i = 0; i < C; ++i)
      if (t0 + i < t_end) v[i] *= __ldg(g.x_scale + t0 + i) * ws;
  }
#pragma unroll
  for (int i = 0; i < C; ++i) v[i] += bias;
  apply_act(v, g.act);
#pragma unroll
  for (int i = 0; i < C; ++i)
    if (t0 + i < t_end) store_typed(g.out, g.out_dt, (t0 + i) * g.ldo + n, v[i] + r[i]);
}

template <int BN, bool FP8>
__global__ void __launch_bounds__(kSplitThreads)
    k_linear_split(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                   const LinearArgs g, int S) {
  using L = SplitCfg<BN>;
  constexpr int KE = FP8 ? 128 : 64;  // K elements per atom
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBarOffset);
  uint64_t* empty = full + L::kStages;
  uint64_t* done = empty + L::kStages;
  uint64_t* drain = done + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = static_cast<int>(blockIdx.x) % S;  // clusters are S consecutive CTAs
  const int tile = static_cast<int>(blockIdx.x) / S;
  const int nt = tile / g.n_tb;
  const int t_base = (tile - nt * g.n_tb) * BN;
  const int k0 = static_cast<int>(static_cast<long long>(g.nk) * rank / S);
  const int k1 = static_cast<int>(static_cast<long long>(g.nk) * (rank + 1) / S);

  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, L::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      // weights pass once through L2 when one token block reads them
      const uint64_t pol_w = g.n_tb == 1 ? policy_evict_first() : policy_evict_last();
      const uint64_t pol_x = policy_evict_last();
      int stage = 0;
      uint32_t phase = 0;
      uint32_t pending = 0, parity = 0;  // stages armed and not re-acquired, for the drain
      bool ok = true;
      for (int k = k0; k < k1; ++k) {
        ok = mbar_wait(&empty[stage], phase ^ 1u, abort_flag);
        if (!ok) break;
        uint8_t* a = smem + stage * L::kStageBytes;
        mbar_arrive_expect_tx(&full[stage], L::kStageBytes);
        tma_load_2d(a, &tmW, &full[stage], k * KE, nt * kTileM, pol_w);
        tma_load_2d(a + kTileM * kTileKBytes, &tmX, &full[stage], k * KE, t_base, pol_x);
        pending |= 1u << stage;
        parity = (parity & ~(1u << stage)) | (phase << stage);
        if (++stage == L::kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) {
        for (int s = 0; s < L::kStages; ++s)
          if ((pending >> s) & 1u) drain_wait(&full[s], (parity >> s) & 1u);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = FP8 ? idesc_e4m3(kTileM, BN) : idesc_16bit(kTileM, BN, g.f16);
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int k = k0; k < k1; ++k) {
        ok = mbar_wait(&full[stage], phase, abort_flag);
        if (!ok) break;
        tc_fence_after();
        const uint32_t a_addr = smem_u32(smem + stage * L::kStageBytes);
        const uint64_t adesc = sw128_kmajor_desc(a_addr);
        const uint64_t bdesc = sw128_kmajor_desc(a_addr + kTileM * kTileKBytes);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {  // 32 K-bytes per MMA: +2 in the (addr >> 4) field
          const uint32_t accum = (k != k0 || kk != 0) ? 1u : 0u;
          if (FP8) umma_f8(tmem_base, adesc + 2 * kk, bdesc + 2 * kk, idesc, accum);
          else umma_f16(tmem_base, adesc + 2 * kk, bdesc + 2 * kk, idesc, accum);
        }
        umma_commit(&empty[stage]);
        if (++stage == L::kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (ok) {
        umma_commit(done);
      } else {
        umma_commit(drain);
        drain_wait(drain, 0);
      }
    }
    __syncwarp();
  }

  const int q = warp & 3;  // TMEM lane quarter of an epilogue warp
  const int rowi = 32 * q + lane;
  const int n = nt * kTileM + rowi;
  const int nv = min(BN, g.T - t_base);  // tokens of this block
  float ws = 0.f, bias = 0.f;
  bool ok = false;
  if (warp >= 2) {
    if (n < g.N) {  // fetched while the sum is still being built
      if (g.x_scale) ws = __ldg(g.w_scale + static_cast<size_t>(n) * g.w_scale_step);
      if (g.bias) bias = load_typed(g.bias, g.bias_dt, n);
    }
    ok = mbar_wait(done, 0, abort_flag);
    __syncwarp();
    tc_fence_after();
  }
  const uint32_t t_row = tmem_base + (static_cast<uint32_t>(32 * q) << 16);
  if (S == 1) {
    if (warp >= 2 && __all_sync(0xffffffffu, ok)) {
      for (int c0 = 0; c0 < nv; c0 += 16) {
        float v[16];
        tmem_ld16(t_row + static_cast<uint32_t>(c0), v);
        tmem_wait_ld();
        if (n < g.N) split_finish<16>(g, v, n, t_base + c0, t_base + nv, ws, bias);
      }
    }
  } else {
    // the stages are free: every copy has landed and every MMA has read them
    float* part = reinterpret_cast<float*>(smem);  // [token column][128 outputs]
    if (warp >= 2 && __all_sync(0xffffffffu, ok)) {
      for (int c0 = 0; c0 < nv; c0 += 16) {
        float v[16];
        tmem_ld16(t_row + static_cast<uint32_t>(c0), v);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) part[(c0 + i) * kTileM + rowi] = v[i];
      }
    }
    cluster_sync_all();
    if (warp >= 2) {
      constexpr int C = 4;
      const int c_lo = nv * rank / S, c_hi = nv * (rank + 1) / S;
      const uint32_t part0 = smem_u32(part) + 4u * static_cast<uint32_t>(rowi);
      for (int c0 = c_lo; c0 < c_hi; c0 += C) {
        float v[C];
#pragma unroll
        for (int i = 0; i < C; ++i) v[i] = 0.f;
        for (int p = 0; p < S; ++p) {
          const uint32_t peer = mapa_shared(part0, static_cast<uint32_t>(p));
#pragma unroll
          for (int i = 0; i < C; ++i)
            if (c0 + i < c_hi) v[i] += ld_shared_cluster_f32(peer + static_cast<uint32_t>((c0 + i) * kTileM * 4));
        }
        if (n < g.N) split_finish<C>(g, v, n, t_base + c0, t_base + c_hi, ws, bias);
      }
    }
    cluster_sync_all();  // no CTA leaves while a peer may still read its partial tile
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, L::kTmemCols);
  }
}

}  // namespace moe
