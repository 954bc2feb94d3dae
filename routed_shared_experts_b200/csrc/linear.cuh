// linear.cuh - dense matrix product with a fused epilogue on tcgen05.
//
//   y[t, n] = round( act( x_scale[t] * w_scale[n] * sum_k x[t, k] w[n, k] + bias[n] ) + residual[t, n] )
//
// x [T, K] and w [N, K] are read by TMA in 128-byte K atoms (64 values of 16
// bits, 128 of 8; the tensor map zero-fills past K, T and N, so any T, N and K
// runs), the sum is kept in fp32 in TMEM, everything after it happens in
// registers, and the result is rounded once. The scales are applied one after
// the other: their own product could leave the fp32 range where the result does
// not.
//
// A pipeline stage holds kLinAtoms K atoms, and two producer warps load one
// operand each, with one copy per stage: the map views the operand as
// [atoms][rows][128 bytes], so that a box of several atoms lands as whole
// swizzled tiles one after another. With one atom per stage and one producer
// each role's fixed cost per stage (barrier wait, arrival, copy issue, commit)
// set the pace, 0.3 us per atom whatever its bytes. The last stage, where K
// ends inside it, is loaded atom by atom through a plain 2D map.
//
// k_linear_split: weights on the MMA's M side (128 outputs per tile), up to BN
// tokens on N, and the K axis split over the S CTAs of a cluster. Each CTA
// leaves its fp32 partial tile in its own shared memory; after a cluster
// barrier every CTA adds the S partials of its share of the token columns over
// distributed shared memory, its own first and the others in a fixed order, and
// finishes them. No workspace, no atomics: the result does not depend on the
// order in which CTAs finish.
// What bounds it: with few tokens the weights' stream from HBM, N * K * size
// bytes, which needs all SMs pulling at once; the K split is what supplies them
// when N / 128 tiles are fewer than the SMs (32 tokens, 7168 x 7168 with
// residual: 19.8 us, 5.3 TB/s, 81 % of the measured copy rate; the library's
// product alone 25.9). Below about 10 MB of weights it is bound by latency: 4.4
// us for one token against 2048 x 2048.
#pragma once
#include <type_traits>

#include "gemm.cuh"
#include "norm.cuh"
#include "ptx_ext.cuh"
#include "router.cuh"

namespace moe {

enum LinearAct : int { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4, kActSigmoid = 5 };

constexpr int kLinAtoms = 2;  // K atoms per pipeline stage

struct LinearArgs {
  int T, N;
  int nk;                // K atoms
  int nk_full;           // of those, atoms that K fills
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
  int n_tb;    // k_linear_tile: 256-token tiles
  int tn, n_nt;  // k_linear_tile: outputs per tile (a multiple of 32, at most 256), tiles along N
  int split;     // k_linear_tile with SPLIT: pairs along K
  int out_unit, res_unit;  // k_linear_tile with SPLIT: bytes that divide every row's address and length: 16, 8, 4 or 2
};

// Instruction descriptor of kind::f16 with both operands bf16 or both fp16.
__host__ __device__ constexpr uint32_t idesc_16bit(int M, int N, bool f16) {
  return f16 ? idesc_bf16(M, N) & ~((7u << 7) | (7u << 10)) : idesc_bf16(M, N);
}

// num * sigmoid(v). ACCURATE (fp32 results): by e = exp(-|v|) in (0, 1], so that
// nothing overflows and the left tail keeps its relative precision down to the
// subnormals; the library's expf (2^-22) and a division by 1 + e in [1, 2] (2^-22)
// leave 2^-20 with the roundings beside them. Else (16-bit results) num / (1 + exp(-v))
// with the fast exponential, ex2 of the rounded product v log2(e): (4 + 1.2 |v|) 2^-23,
// far below the store's half step, and zeros in place of results below 2^-119, where
// the fast division's divisor passes 2^126. The accurate form costs fp32 results 2 to
// 8 % (4096 x 256 x 7168 SiLU 23.0 -> 23.5 us, 777 x 2815 x 4096 tanh-GELU 38.5 ->
// 41.7) and would cost 16-bit ones, whose store hides the difference, 3 %.
template <bool ACCURATE>
__device__ __forceinline__ float times_sigmoid(float num, float v) {
  if (!ACCURATE) return __fdividef(num, 1.0f + __expf(-v));
  const float e = expf(-fabsf(v));
  return num * __fdividef(v < 0.f ? e : 1.0f, 1.0f + e);
}

// The activation of C accumulated values. NaN passes through every one.
template <bool ACCURATE, int C>
__device__ __forceinline__ void apply_act(float (&v)[C], int act) {
  switch (act) {
    case kActRelu:
#pragma unroll
      for (int i = 0; i < C; ++i) v[i] = v[i] < 0.f ? 0.f : v[i];
      break;
    case kActSilu:
#pragma unroll
      for (int i = 0; i < C; ++i) v[i] = times_sigmoid<ACCURATE>(v[i], v[i]);
      break;
    case kActGelu:  // v * Phi(v). erff against erfcf(-x): 23 against 31 us at 777 x 2815 x 4096, for an
                    // absolute error of 2^-24 |v| in the left tail, where the result itself vanishes
#pragma unroll
      for (int i = 0; i < C; ++i) v[i] = 0.5f * v[i] * (1.0f + erff(0.70710678118654752f * v[i]));
      break;
    case kActGeluTanh:  // 0.5 v (1 + tanh u) = v sigmoid(2u)
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const float u2 = 1.5957691216057308f * (v[i] + 0.044715f * v[i] * v[i] * v[i]);
        v[i] = times_sigmoid<ACCURATE>(v[i], u2);
      }
      break;
    case kActSigmoid:
#pragma unroll
      for (int i = 0; i < C; ++i) v[i] = times_sigmoid<ACCURATE>(1.0f, v[i]);
      break;
    default: break;
  }
}

__device__ __forceinline__ float load_typed(const void* p, int dt, size_t i) {
  if (dt == 4) return static_cast<const float*>(p)[i];
  const unsigned short b = static_cast<const unsigned short*>(p)[i];
  return dt == 0 ? __bfloat162float(__ushort_as_bfloat16(b)) : __half2float(__ushort_as_half(b));
}

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

// 0 where `on` is false. A predicate rather than a branch, so that a batch of
// loads goes out together.
__device__ __forceinline__ float ld_shared_cluster_f32_if(uint32_t cluster_addr, bool on) {
  float v;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %2, 0;\n\t"
      "mov.f32 %0, 0f00000000;\n\t"
      "@p ld.shared::cluster.f32 %0, [%1];\n\t}\n"
      : "=f"(v)
      : "r"(cluster_addr), "r"(static_cast<int>(on))
      : "memory");
  return v;
}

// Copies of stage `ks` of one operand: rows row0.. into consecutive tiles of
// `atom_bytes`. `tm`: the [atoms][rows][128 bytes] map, `tail`: the 2D map.
template <int KE, bool PAIR>
__device__ __forceinline__ void load_stage(uint8_t* dst, const CUtensorMap* tm, const CUtensorMap* tail, uint64_t* bar,
                                           uint32_t bar_cluster, int ks, int row0, int atom_bytes, const LinearArgs& g,
                                           uint64_t policy) {
  const int k0 = ks * kLinAtoms;
  if (k0 + kLinAtoms <= g.nk_full) {
    if constexpr (PAIR) tma_load_3d_pair(dst, tm, bar_cluster, 0, row0, k0, policy);
    else tma_load_3d(dst, tm, bar, 0, row0, k0, policy);
  } else {
#pragma unroll
    for (int a = 0; a < kLinAtoms; ++a) {
      if (k0 + a < g.nk) {
        if constexpr (PAIR) tma_load_2d_pair(dst + a * atom_bytes, tail, bar_cluster, (k0 + a) * KE, row0, policy);
        else tma_load_2d(dst + a * atom_bytes, tail, bar, (k0 + a) * KE, row0, policy);
      }
    }
  }
}

// Uses of accumulator `acc` (0 or 1) in `n` accumulations that take turns.
__host__ __device__ constexpr int acc_uses(int n, int acc) { return (n + 1 - acc) / 2; }
// Parity whose wait ends with the release that follows an accumulator's last use.
__host__ __device__ constexpr uint32_t last_release_parity(int uses) { return static_cast<uint32_t>(uses - 1) & 1u; }

// ------------------------------------------------------------ K split over a cluster

constexpr int kSplitThreads = 224;  // weight producer, MMA, token producer, four epilogue warps
constexpr int kSplitPieceStages = 7;  // 14 atoms: the longest accumulation of an fp32 result

template <int BN>
struct SplitCfg {
  static constexpr int kAtomW = kTileM * kTileKBytes;
  static constexpr int kAtomX = BN * kTileKBytes;
  static constexpr int kStageBytes = (kAtomW + kAtomX) * kLinAtoms;
  static constexpr int kMaxStages = 6;
  static constexpr int kStageOffset = 1024;  // after the barriers
  // TMEM columns: two accumulators with PROMOTE, so that two CTAs on an SM hold 256 of the 512 at most
  __host__ __device__ static constexpr int tmem_cols(bool promote) { return promote ? 2 * BN : BN < 32 ? 32 : BN; }
  static_assert(kStageBytes % 1024 == 0, "stages start on 1024-byte swizzle boundaries");
  static_assert((2 * kMaxStages + 5) * 8 + 8 <= kStageOffset, "barriers");
  // as many stages as fit `bytes` of shared memory (one CTA per SM, or two)
  __host__ __device__ static constexpr int stages(int bytes) {
    const int fit = (bytes - 1024 - kStageOffset) / kStageBytes;  // less the alignment slack
    return fit < kMaxStages ? fit : kMaxStages;
  }
  __host__ __device__ static constexpr int bytes(int n_stages) { return kStageOffset + n_stages * kStageBytes + 1024; }
  static_assert(BN * kTileM * 4 <= 2 * kStageBytes, "the partial tile fits the stages it replaces");
};

// A thread's output n of the split kernel: its tokens are finished in batches of
// 16, or 8 where no more are left, so that a batch's remote loads and residual
// loads are in flight together and one token does not pay for sixteen (with
// residual, K = 7168: 22.6 -> 20.6 us for 32 tokens against batches of 8 alone;
// N = 2048, one token: 5.5 us against 6.8 with batches of 16 alone). Tiles of 16
// tokens have no use for the wider batch, whose registers cost them 0.3 us.
// F32: fp32 results, a kernel each, so that the code of one result type is all that a launch
// of a few microseconds fetches.
template <int B, bool F32>  // B: widest batch, 8 or 16
struct SplitOut {
  const LinearArgs& g;
  int n;
  float ws, bias;

  // No condition per value, so that the loads go out together: tokens past t_end
  // read the last one's.
  template <int C>
  __device__ __forceinline__ void residual(float (&r)[B], int t0, int t_end) const {
    if (!g.residual || n >= g.N) {
#pragma unroll
      for (int i = 0; i < C; ++i) r[i] = 0.f;
    } else if (F32) {
      const float* p = static_cast<const float*>(g.residual) + n;
#pragma unroll
      for (int i = 0; i < C; ++i) r[i] = p[min(t0 + i, t_end - 1) * g.ldr];
    } else {
      const unsigned short* p = static_cast<const unsigned short*>(g.residual) + n;
      unsigned short h[C];
#pragma unroll
      for (int i = 0; i < C; ++i) h[i] = p[min(t0 + i, t_end - 1) * g.ldr];
#pragma unroll
      for (int i = 0; i < C; ++i)
        r[i] = g.out_dt == 0 ? __bfloat162float(__ushort_as_bfloat16(h[i])) : __half2float(__ushort_as_half(h[i]));
    }
  }
  __device__ __forceinline__ void residual_of(float (&r)[B], int t0, int t_end) const {
    if (t_end <= t0) return;  // no tokens in this CTA's share
    if (B == 8 || t_end - t0 <= 8) residual<8>(r, t0, t_end);
    else residual<B>(r, t0, t_end);
  }
  // Scale, bias, activation, residual and store of tokens t0 .. t0 + C - 1.
  template <int C>
  __device__ __forceinline__ void finish(float (&v)[C], const float (&r)[B], int t0, int t_end) const {
    if (n >= g.N || t0 >= t_end) return;
    if (g.x_scale) {
      float xs[C];
#pragma unroll
      for (int i = 0; i < C; ++i) xs[i] = g.x_scale[min(t0 + i, t_end - 1)];
#pragma unroll
      for (int i = 0; i < C; ++i) v[i] = v[i] * xs[i] * ws;
    }
#pragma unroll
    for (int i = 0; i < C; ++i) v[i] += bias;
    apply_act<F32>(v, g.act);
    if (F32) {
      float* p = static_cast<float*>(g.out) + t0 * g.ldo + n;
#pragma unroll
      for (int i = 0; i < C; ++i)
        if (t0 + i < t_end) p[i * g.ldo] = v[i] + r[i];
    } else {
      unsigned short* p = static_cast<unsigned short*>(g.out) + t0 * g.ldo + n;
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const float y = v[i] + r[i];
        const unsigned short h = g.out_dt == 0 ? __bfloat16_as_ushort(__float2bfloat16_rn(y))
                                               : __half_as_ushort(__float2half_rn(y));
        if (t0 + i < t_end) p[i * g.ldo] = h;
      }
    }
  }
  // Columns c0 .. c0 + C - 1 of the S partial tiles ([token column][128 outputs];
  // `part`: this thread's output of column 0), this CTA's own first, so that the
  // peers' reads spread. Only what finish() uses is read: the relaxed cluster barrier
  // that ends the kernel does not wait for a load whose value nothing waits for, and a
  // peer could be gone before it arrives.
  template <int C>
  __device__ __forceinline__ void join(uint32_t part, int rank, int S, int c0, int c_hi,
                                       const float (&r)[B]) const {
    float v[C];
#pragma unroll
    for (int i = 0; i < C; ++i) v[i] = 0.f;
    const bool in = n < g.N;
#pragma unroll 2
    for (int p = 0; p < S; ++p) {
      const uint32_t peer = mapa_shared(part, static_cast<uint32_t>((rank + p) & (S - 1)));
#pragma unroll
      for (int i = 0; i < C; ++i)
        v[i] += ld_shared_cluster_f32_if(peer + static_cast<uint32_t>((c0 + i) * kTileM * 4), in && c0 + i < c_hi);
    }
    finish(v, r, c0, c_hi);
  }
};

// PROMOTE: this CTA's share of K is cut into accumulations of kSplitPieceStages stages
// that take turns on two TMEM accumulators; the epilogue threads add them in fp32
// registers. For fp32 results whose K is longer than one such piece for each of
// the 8 CTAs of a cluster (S is 8 then). Positive bf16 values, 64 tokens, K = 57344:
// off by 1.7e-6 of the result, as at K = 7168, against 2.9e-5 in one accumulation per
// CTA; 32 x 2048 x 16384 takes 22.0 us, 22.3 in one accumulation.
template <int BN, bool FP8, bool F32, bool PROMOTE>
__global__ void __launch_bounds__(kSplitThreads)
    k_linear_split(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmWt,
                   const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmXt,
                   const LinearArgs g, int S, int n_stages) {
  using L = SplitCfg<BN>;
  constexpr int KE = FP8 ? 128 : 64;  // K elements per atom
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* stages = smem + L::kStageOffset;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem);
  uint64_t* empty = full + L::kMaxStages;
  uint64_t* acc_full = empty + L::kMaxStages;  // [2] with PROMOTE, else [1]
  uint64_t* acc_empty = acc_full + 2;          // [2], PROMOTE only
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = static_cast<int>(blockIdx.x) % S;  // clusters are S consecutive CTAs
  const int nt = static_cast<int>(blockIdx.x) / S;
  const int ns = (g.nk + kLinAtoms - 1) / kLinAtoms;  // stages along K; this CTA's are s0 .. s1 - 1
  const int s0 = static_cast<int>(static_cast<long long>(ns) * rank / S);
  const int s1 = static_cast<int>(static_cast<long long>(ns) * (rank + 1) / S);
  // accumulations that the share is cut into
  const int n_kc = PROMOTE ? (s1 - s0 + kSplitPieceStages - 1) / kSplitPieceStages : 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < n_stages; ++s) {
      mbar_init(&full[s], 2);  // each producer arms it with its own bytes
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&acc_full[a], 1);
      mbar_init(&acc_empty[a], 4);  // the epilogue warps
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, L::tmem_cols(PROMOTE));
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  grid_dependents_launch();
  grid_dependency_wait();

  if (warp == 0 || warp == 2) {
    if (elect_one()) {
      const bool is_w = warp == 0;
      const CUtensorMap* tm = is_w ? &tmW : &tmX;
      const CUtensorMap* tail = is_w ? &tmWt : &tmXt;
      const uint64_t pol = is_w ? policy_evict_first() : policy_evict_last();  // the weights pass once
      const int row0 = is_w ? nt * kTileM : 0;
      const int atom_bytes = is_w ? L::kAtomW : L::kAtomX;
      const int off = is_w ? 0 : L::kAtomW * kLinAtoms;
      int stage = 0;
      uint32_t phase = 0;
      uint32_t pending = 0, parity = 0;  // stages armed and not re-acquired, for the drain
      bool ok = true;
      for (int ks = s0; ks < s1; ++ks) {
        ok = mbar_wait(&empty[stage], phase ^ 1u, abort_flag);
        if (!ok) break;
        const int na = min(kLinAtoms, g.nk - ks * kLinAtoms);
        mbar_arrive_expect_tx(&full[stage], static_cast<uint32_t>(na * atom_bytes));
        load_stage<KE, false>(stages + stage * L::kStageBytes + off, tm, tail, &full[stage], 0, ks, row0, atom_bytes, g,
                              pol);
        pending |= 1u << stage;
        parity = (parity & ~(1u << stage)) | (phase << stage);
        if (++stage == n_stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) {
        for (int s = 0; s < n_stages; ++s)
          if ((pending >> s) & 1u) drain_wait(&full[s], (parity >> s) & 1u);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (elect_one()) {
      const uint32_t idesc = FP8 ? idesc_e4m3(kTileM, BN) : idesc_16bit(kTileM, BN, g.f16);
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int kc = 0; kc < n_kc && ok; ++kc) {
        const int acc = PROMOTE ? kc & 1 : 0;
        if (PROMOTE) {
          ok = mbar_wait(&acc_empty[acc], ((static_cast<uint32_t>(kc) >> 1) & 1u) ^ 1u, abort_flag);
          if (!ok) break;
          tc_fence_after();
        }
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * BN);
        const int s_lo = PROMOTE ? s0 + kc * kSplitPieceStages : s0;
        const int s_hi = PROMOTE ? min(s1, s_lo + kSplitPieceStages) : s1;
        for (int ks = s_lo; ks < s_hi; ++ks) {
          ok = mbar_wait(&full[stage], phase, abort_flag);
          if (!ok) break;
          tc_fence_after();
          const int na = min(kLinAtoms, g.nk - ks * kLinAtoms);
          const uint32_t a_addr = smem_u32(stages + stage * L::kStageBytes);
#pragma unroll
          for (int a = 0; a < kLinAtoms; ++a) {
            if (a < na) {
              const uint64_t adesc = sw128_kmajor_desc(a_addr + a * L::kAtomW);
              const uint64_t bdesc = sw128_kmajor_desc(a_addr + L::kAtomW * kLinAtoms + a * L::kAtomX);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) {  // 32 K-bytes per MMA: +2 in the (addr >> 4) field
                const uint32_t accum = (ks != s_lo || (a | kk) != 0) ? 1u : 0u;
                if (FP8) umma_f8(d_tmem, adesc + 2 * kk, bdesc + 2 * kk, idesc, accum);
                else umma_f16(d_tmem, adesc + 2 * kk, bdesc + 2 * kk, idesc, accum);
              }
            }
          }
          if (ks + n_stages < s1) umma_commit(&empty[stage]);  // a release that no refill waits for is not sent
          if (++stage == n_stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (ok) umma_commit(&acc_full[acc]);
      }
      if (!ok) {
        umma_commit(drain);
        drain_wait(drain, 0);
      }
    }
    __syncwarp();
  }

  const int q = warp & 3;  // TMEM lane quarter of an epilogue warp
  const int rowi = 32 * q + lane;
  const int n = nt * kTileM + rowi;
  const int nv = min(BN, g.T);  // tokens
  // S > 1: this CTA finishes columns c_lo .. c_hi - 1
  const int c_lo = nv * rank / S, c_hi = nv * (rank + 1) / S;
  constexpr int B = BN == 16 ? 8 : 16;
  SplitOut<B, F32> o{g, n, 0.f, 0.f};
  float res[B];
  bool ok = false;
  if (warp >= 3) {
    if (n < g.N) {  // fetched while the sum is still being built
      if (g.x_scale) o.ws = g.w_scale[static_cast<size_t>(n) * g.w_scale_step];
      if (g.bias) o.bias = load_typed(g.bias, g.bias_dt, n);
    }
    o.residual_of(res, c_lo, c_hi);
  }
  const uint32_t t_row = tmem_base + (static_cast<uint32_t>(32 * q) << 16);
  float sum[PROMOTE ? BN : 1];
  if (warp >= 3) {
    for (int kc = 0; kc < n_kc; ++kc) {
      const int acc = kc & 1;
      ok = mbar_wait(&acc_full[acc], (static_cast<uint32_t>(kc) >> 1) & 1u, abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      if constexpr (PROMOTE) {
#pragma unroll
        for (int c0 = 0; c0 < BN; c0 += 16) {
          float v[16];
          tmem_ld16(t_row + static_cast<uint32_t>(acc * BN + c0), v);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) sum[c0 + i] = kc == 0 ? v[i] : sum[c0 + i] + v[i];
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty[acc]);
      }
    }
  }
  if (!PROMOTE && S == 1) {
    if (ok) {
      for (int c0 = 0; c0 < nv; c0 += 16) {
        float v[16];
        tmem_ld16(t_row + static_cast<uint32_t>(c0), v);
        tmem_wait_ld();
#pragma unroll
        for (int h = 0; h < 16 / B; ++h) {
          const int t0 = c0 + B * h;
          float u[B];
#pragma unroll
          for (int i = 0; i < B; ++i) u[i] = v[B * h + i];
          if (c0 + h > 0) o.residual_of(res, t0, nv);
          o.finish(u, res, t0, nv);
        }
      }
    }
  } else {
    // the stages are free: every copy has landed and every MMA has read them
    float* part = reinterpret_cast<float*>(stages);  // [token column][128 outputs]
    if (PROMOTE && ok) {
#pragma unroll
      for (int c = 0; c < BN; ++c) part[c * kTileM + rowi] = sum[PROMOTE ? c : 0];
    } else if (ok) {
      for (int c0 = 0; c0 < nv; c0 += 16) {
        float v[16];
        tmem_ld16(t_row + static_cast<uint32_t>(c0), v);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) part[(c0 + i) * kTileM + rowi] = v[i];
      }
    }
    cluster_sync_all();
    if (warp >= 3) {
      const uint32_t part0 = smem_u32(part) + 4u * static_cast<uint32_t>(rowi);
      for (int c0 = c_lo; c0 < c_hi;) {
        if (c0 > c_lo) o.residual_of(res, c0, c_hi);
        if (B == 8 || c_hi - c0 <= 8) {
          o.template join<8>(part0, rank, S, c0, c_hi, res);
          c0 += 8;
        } else {
          o.template join<B>(part0, rank, S, c0, c_hi, res);
          c0 += B;
        }
      }
    }
    cluster_sync_relaxed();  // no CTA leaves while a peer may still read its partial tile
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, L::tmem_cols(PROMOTE));
  }
}

// ------------------------------------------------------------ CTA pairs, many tokens
//
// k_linear_tile: a 2-CTA cluster per tile of 256 tokens (M, 128 in each CTA)
// x tn outputs (N, tn / 2 weight rows in each CTA), persistent over the tiles.
// Warps 0 and 2 load (tokens and weights, each CTA its half of both), rank 0's
// warp 1 issues the pair's MMAs, and eight epilogue warps per CTA empty one TMEM
// accumulator while the MMAs fill the other. tn is chosen by the host so that the
// tiles fill whole waves of pairs. Each epilogue warp owns 32 token rows and
// turns its columns, 32 at a time, through 2 KB of shared memory, so that
// residual reads and result writes are whole 64-byte row segments and no barrier
// between warps is needed.
//
// What bounds it: wide tiles by the MMAs (at tn = 256 a stage of two atoms takes
// 1023 of the ideal 1024 clocks; T = 4096, N = K = 7168 runs at 224 outputs, tensor
// pipe 89 % busy) and, kept up, by the 1 kW power cap: that product with residual
// takes 306 us from a cool start and 348 sustained at 1.2 GHz, 1.21 PFLOP/s against
// 1.38 measured sustained (the library's product alone, in turn with it: 314 and
// 360). Narrow tiles wait for their copies, whose round trip of
// about 1.45 us the stages that fit have to cover: hence as many as fit. Small
// shapes are bound by what a launch, the first copy and the last tile's epilogue
// take, 5 to 7 us.
//
// SPLIT: the K axis of a tile is divided over the `split` pairs of one cluster,
// for shapes whose tiles are fewer than the pairs of SMs. As in k_linear_split
// each CTA leaves its fp32 partial tile in its own shared memory and the CTAs of
// the same token half finish 128 / split rows each, adding the partials over
// distributed shared memory in a fixed order.
//
// PROMOTE (fp32 results): the tensor core's accumulation is cut every
// kPromoteAtoms K atoms and the pieces are added in registers in fp32 (round
// to nearest), which the accumulator's own additions are not: one accumulation
// of 1792 values was off by 1.7e-6 of the sum's rms and the error grows with their
// number; K = 7168 in pieces is off by 0.5e-6. A 16-bit result's rounding hides
// that error, so those keep one accumulation. With SPLIT the pieces are the two
// halves of a pair's share of K, one in each accumulator.

constexpr int kTileEpiWarps = 8;
constexpr int kTileThreads = 96 + 32 * kTileEpiWarps;  // two producers, MMA, epilogue
constexpr int kPromoteAtoms = 8;
constexpr int kPromoteTn = 128;  // outputs per tile with PROMOTE: 64 running sums per epilogue thread

struct TileCfg {
  static constexpr int kMaxStages = 5;
  static constexpr int kAtom = kTileM * kTileKBytes;
  static constexpr int kABytes = kAtom * kLinAtoms;  // 128 tokens
  static constexpr int kWarpOut = 2048;              // 32 rows x 64 bytes
  static constexpr int kBarOffset = kTileEpiWarps * kWarpOut;
  static constexpr int kStageOffset = kBarOffset + 1024;
  static constexpr int kTmemCols = 512;
  static_assert((2 * kMaxStages + 5) * 8 + 8 <= 1024, "barriers");
  // a stage: 128 tokens, then tn / 2 weight rows, of kLinAtoms atoms
  __host__ __device__ static constexpr int stage_bytes(int tn) { return kABytes + tn / 2 * kTileKBytes * kLinAtoms; }
  __host__ __device__ static constexpr int stages(int tn) {
    const int fit = (227 * 1024 - 1024 - kStageOffset) / stage_bytes(tn);  // less the alignment slack
    return fit < kMaxStages ? fit : kMaxStages;
  }
  __host__ __device__ static constexpr int bytes(int tn) { return kStageOffset + stages(tn) * stage_bytes(tn) + 1024; }
};

// Byte offset of 16-byte unit u of row r in a warp's 32 x 64-byte staging: the
// XOR spreads both the row-wise and the row-group-wise accesses over all banks.
__device__ __forceinline__ int stage_off(int r, int u) { return r * 64 + ((u ^ ((r >> 1) & 3)) << 4); }

// A warp's copies between 32 rows of a matrix, 64 bytes each (`bytes` of them
// valid, `rows` rows valid), and its staging, in units of U = 16, 8, 4 or 2
// bytes: 64 / U lanes take a row, so a copy instruction moves whole row segments
// whatever their alignment. A lane's registers hold its units of rows
// lane * U / 64, + 32 U / 64, ... one after another (U = 2: two to a register).
// Whole segments are copied without conditions, so that the loads go out together.
template <int U>
using unit_t = std::conditional_t<
    U == 16, uint4, std::conditional_t<U == 8, uint2, std::conditional_t<U == 4, uint32_t, unsigned short>>>;

template <int U>
__device__ __forceinline__ void fetch_rows(uint32_t (&v)[16], const uint8_t* src, size_t ld, int rows, int bytes,
                                           int lane) {
  constexpr int kLanes = 64 / U, kRows = 32 / kLanes;  // lanes per row, rows per instruction
  const int at = lane % kLanes * U, r0 = lane / kLanes;
  unit_t<U> f[kLanes];
  src += r0 * ld + at;
  if (rows >= 32 && bytes == 64) {
#pragma unroll
    for (int i = 0; i < kLanes; ++i) f[i] = *reinterpret_cast<const unit_t<U>*>(src + kRows * i * ld);
  } else {
#pragma unroll
    for (int i = 0; i < kLanes; ++i) {
      f[i] = unit_t<U>{};
      if (kRows * i + r0 < rows && at < bytes) f[i] = *reinterpret_cast<const unit_t<U>*>(src + kRows * i * ld);
    }
  }
#pragma unroll
  for (int i = 0; i < kLanes; ++i) {
    if constexpr (U == 16) v[4 * i] = f[i].x, v[4 * i + 1] = f[i].y, v[4 * i + 2] = f[i].z, v[4 * i + 3] = f[i].w;
    else if constexpr (U == 8) v[2 * i] = f[i].x, v[2 * i + 1] = f[i].y;
    else if constexpr (U == 4) v[i] = f[i];
    else if (i % 2 == 0) v[i / 2] = f[i] | (static_cast<uint32_t>(f[i + 1]) << 16);
  }
}

template <int U>
__device__ __forceinline__ void stage_put(uint8_t* st, const uint32_t (&v)[16], int lane) {
  constexpr int kLanes = 64 / U, kRows = 32 / kLanes;
  const int at = lane % kLanes * U, r0 = lane / kLanes;
#pragma unroll
  for (int i = 0; i < kLanes; ++i) {
    uint8_t* to = st + stage_off(kRows * i + r0, at >> 4) + (at & 15);
    if constexpr (U == 16)
      *reinterpret_cast<uint4*>(to) = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    else if constexpr (U == 8) *reinterpret_cast<uint2*>(to) = make_uint2(v[2 * i], v[2 * i + 1]);
    else if constexpr (U == 4) *reinterpret_cast<uint32_t*>(to) = v[i];
    else *reinterpret_cast<unsigned short*>(to) = static_cast<unsigned short>(v[i / 2] >> (16 * (i % 2)));
  }
}

template <int U>
__device__ __forceinline__ void stage_store(const uint8_t* st, uint8_t* dst, size_t ld, int rows, int bytes, int lane) {
  constexpr int kLanes = 64 / U, kRows = 32 / kLanes;
  const int at = lane % kLanes * U, r0 = lane / kLanes;
  unit_t<U> v[kLanes];  // all read before any is stored
#pragma unroll
  for (int i = 0; i < kLanes; ++i)
    v[i] = *reinterpret_cast<const unit_t<U>*>(st + stage_off(kRows * i + r0, at >> 4) + (at & 15));
  dst += r0 * ld + at;
  if (rows >= 32 && bytes == 64) {
#pragma unroll
    for (int i = 0; i < kLanes; ++i) *reinterpret_cast<unit_t<U>*>(dst + kRows * i * ld) = v[i];
  } else if (at < bytes) {
#pragma unroll
    for (int i = 0; i < kLanes; ++i)
      if (kRows * i + r0 < rows) *reinterpret_cast<unit_t<U>*>(dst + kRows * i * ld) = v[i];
  }
}

// Valid bytes of a row's 64 from column n0 < N on. Counted in columns first: N - n0
// times the value's size passes 31 bits from N = 2^29 (fp32) on.
template <int OS>
__host__ __device__ constexpr int chunk_bytes(int N, int n0) {
  return (N - n0 < 64 / OS ? N - n0 : 64 / OS) * OS;
}

// Residual rows of this warp from column n0 (64 bytes of each; OS: bytes of a value).
template <int OS, int U>
__device__ __forceinline__ void fetch_residual(const LinearArgs& g, uint32_t (&v)[16], int row0, int n0, int lane) {
  fetch_rows<U>(v, static_cast<const uint8_t*>(g.residual) + (row0 * g.ldr + n0) * OS, g.ldr * OS, g.T - row0,
                chunk_bytes<OS>(g.N, n0), lane);
}

template <int OS, int U>
__device__ __forceinline__ void store_result(const LinearArgs& g, const uint8_t* st, int row0, int n0, int lane) {
  stage_store<U>(st, static_cast<uint8_t*>(g.out) + (row0 * g.ldo + n0) * OS, g.ldo * OS, g.T - row0,
                 chunk_bytes<OS>(g.N, n0), lane);
}

// Residual, rounding and store of 32 columns n0.. of this warp's 32 rows
// (16-bit results): thread = row, through the staging. `res`: the residual
// fetched ahead (fetch_residual).
template <typename TX, int U>
__device__ __forceinline__ void tile_store_16(const LinearArgs& g, uint8_t* st, float (&v)[32],
                                              const uint32_t (&res)[16], int row0, int n0, int lane) {
  if (g.residual) {
    stage_put<U>(st, res, lane);
    __syncwarp();
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      float f[8];
      unpack8<TX>(*reinterpret_cast<const uint4*>(st + stage_off(lane, u)), f);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[8 * u + i] += f[i];
    }
  }
#pragma unroll
  for (int u = 0; u < 4; ++u)
    *reinterpret_cast<uint4*>(st + stage_off(lane, u)) =
        make_uint4(pack2(v[8 * u], v[8 * u + 1], TX()), pack2(v[8 * u + 2], v[8 * u + 3], TX()),
                   pack2(v[8 * u + 4], v[8 * u + 5], TX()), pack2(v[8 * u + 6], v[8 * u + 7], TX()));
  __syncwarp();
  store_result<2, U>(g, st, row0, n0, lane);
  __syncwarp();  // the staging is rewritten next
}

// The same with fp32 results: two halves of 16 columns (`res`: the first one's).
template <int U>
__device__ __forceinline__ void tile_store_32(const LinearArgs& g, uint8_t* st, float (&v)[32], uint32_t (&res)[16],
                                              int row0, int n0, int lane) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int c0 = n0 + 16 * h;
    if (c0 >= g.N) return;
    if (g.residual) {
      stage_put<U>(st, res, lane);
      if (h == 0 && c0 + 16 < g.N) fetch_residual<4, U>(g, res, row0, c0 + 16, lane);  // the second half, meanwhile
      __syncwarp();
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float4 f = *reinterpret_cast<const float4*>(st + stage_off(lane, u));
        v[16 * h + 4 * u] += f.x;
        v[16 * h + 4 * u + 1] += f.y;
        v[16 * h + 4 * u + 2] += f.z;
        v[16 * h + 4 * u + 3] += f.w;
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      *reinterpret_cast<float4*>(st + stage_off(lane, u)) =
          make_float4(v[16 * h + 4 * u], v[16 * h + 4 * u + 1], v[16 * h + 4 * u + 2], v[16 * h + 4 * u + 3]);
    __syncwarp();
    store_result<4, U>(g, st, row0, c0, lane);
    __syncwarp();
  }
}

// Token tile and output tile of `tile`: bands of 8 token tiles, tokens fastest,
// so that the pairs running at one time share operand rows in L2.
__device__ __forceinline__ void tile_coords(const LinearArgs& g, int tile, int& mt, int& nt) {
  constexpr int kBand = 8;
  const int per_band = kBand * g.n_nt;
  const int band = tile / per_band;
  const int rows = min(kBand, g.n_tb - band * kBand);
  const int i = tile - band * per_band;
  nt = i / rows;
  mt = band * kBand + (i - nt * rows);
}

// SPLIT: rows [lo, hi) of this CTA's 128 from the S partial tiles, a warp per two
// rows, four columns per lane. A partial tile is [128][tn] fp32 in 16-byte units,
// unit u of row r at u ^ (r & 7).
__device__ __forceinline__ int part_unit(int r, int u, int tn) { return r * (tn / 4) + (u ^ (r & 7)); }

// Zeros where `on` is false.
__device__ __forceinline__ float4 ld_shared_cluster_f32x4_if(uint32_t cluster_addr, bool on) {
  float4 v;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "mov.f32 %0, 0f00000000;\n\tmov.f32 %1, 0f00000000;\n\t"
      "mov.f32 %2, 0f00000000;\n\tmov.f32 %3, 0f00000000;\n\t"
      "@p ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];\n\t}\n"
      : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
      : "r"(cluster_addr), "r"(static_cast<int>(on))
      : "memory");
  return v;
}

// Four consecutive values (`cols` of them valid) of the residual and the result.
__device__ __forceinline__ void load_res4(const LinearArgs& g, size_t at, int cols, float (&res)[4]) {
  if (g.res_unit == 16 && cols == 4) {
    if (g.out_dt == 4) {
      const float4 f = *reinterpret_cast<const float4*>(static_cast<const float*>(g.residual) + at);
      res[0] = f.x, res[1] = f.y, res[2] = f.z, res[3] = f.w;
    } else {
      const uint2 f = *reinterpret_cast<const uint2*>(static_cast<const unsigned short*>(g.residual) + at);
      if (g.out_dt == 0) {
        unpack2(f.x, __nv_bfloat16(), res[0], res[1]);
        unpack2(f.y, __nv_bfloat16(), res[2], res[3]);
      } else {
        unpack2(f.x, __half(), res[0], res[1]);
        unpack2(f.y, __half(), res[2], res[3]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < cols) res[i] = load_residual(g.residual, g.out_dt, at + i);
  }
}

__device__ __forceinline__ void store4(const LinearArgs& g, size_t at, int cols, const float (&v)[4]) {
  if (g.out_unit == 16 && cols == 4) {
    if (g.out_dt == 4)
      *reinterpret_cast<float4*>(static_cast<float*>(g.out) + at) = make_float4(v[0], v[1], v[2], v[3]);
    else if (g.out_dt == 0)
      *reinterpret_cast<uint2*>(static_cast<unsigned short*>(g.out) + at) =
          make_uint2(pack2(v[0], v[1], __nv_bfloat16()), pack2(v[2], v[3], __nv_bfloat16()));
    else
      *reinterpret_cast<uint2*>(static_cast<unsigned short*>(g.out) + at) =
          make_uint2(pack2(v[0], v[1], __half()), pack2(v[2], v[3], __half()));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < cols) store_typed(g.out, g.out_dt, at + i, v[i]);
  }
}

template <bool F32>
__device__ __forceinline__ void split_rows(const LinearArgs& g, uint32_t part, uint32_t ctarank, int mt, int nt, int ew,
                                           int lane) {
  const int S = g.split;
  const int lo = kTileM / S * static_cast<int>(ctarank >> 1), hi = lo + kTileM / S;
  const int t0 = mt * 2 * kTileM + static_cast<int>(ctarank & 1u) * kTileM;
  for (int u = lane; u < g.tn / 4; u += 32) {
    const int n = nt * g.tn + 4 * u;
    const int cols = min(4, g.N - n);
    if (cols <= 0) continue;
    float ws[4], bias[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      ws[i] = g.w_scale && i < cols ? g.w_scale[static_cast<size_t>(n + i) * g.w_scale_step] : 1.f;
      bias[i] = g.bias && i < cols ? load_typed(g.bias, g.bias_dt, n + i) : 0.f;
    }
    // two rows at a time: their remote loads are in flight together
    constexpr int R = 2;
    for (int r0 = lo + R * ew; r0 < hi && t0 + r0 < g.T; r0 += R * kTileEpiWarps) {
      float res[R][4], v[R][4], xs[R];
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const int t = t0 + r0 + j;
        const bool in = t < g.T;
        xs[j] = g.x_scale && in ? g.x_scale[t] : 1.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[j][i] = res[j][i] = 0.f;
        if (g.residual && in) load_res4(g, t * g.ldr + n, cols, res[j]);
      }
#pragma unroll 2
      for (int p = 0; p < S; ++p) {  // from this CTA's own partial tile on, so that the peers' reads spread
        const uint32_t peer = mapa_shared(part, (ctarank + 2u * static_cast<uint32_t>(p)) & (2u * S - 1u));
#pragma unroll
        for (int j = 0; j < R; ++j) {
          // rows past T are not read: no load may be in flight when a peer ends (as in SplitOut::join)
          const float4 f = ld_shared_cluster_f32x4_if(
              peer + 16u * static_cast<uint32_t>(part_unit(r0 + j, u, g.tn)), t0 + r0 + j < g.T);
          v[j][0] += f.x;
          v[j][1] += f.y;
          v[j][2] += f.z;
          v[j][3] += f.w;
        }
      }
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const int t = t0 + r0 + j;
        if (t >= g.T) break;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[j][i] = v[j][i] * xs[j] * ws[i] + bias[i];
        apply_act<F32>(v[j], g.act);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[j][i] += res[j][i];
        store4(g, t * g.ldo + n, cols, v[j]);
      }
    }
  }
}

// U: the unit of the result's and the residual's rows, a kernel each: one kernel
// that chose among them ran out of registers (4096 x 7168 x 512: 41.3 against
// 36.4 us). SPLIT goes by g.out_unit and g.res_unit instead.
template <bool FP8, bool PROMOTE, bool SPLIT, int U>
__global__ void __launch_bounds__(kTileThreads, 1)
    k_linear_tile(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmXt,
                  const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmWt,
                  const LinearArgs g) {
  using L = TileCfg;
  constexpr int KE = FP8 ? 128 : 64;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBarOffset);
  uint64_t* empty = full + L::kMaxStages;
  uint64_t* acc_full = empty + L::kMaxStages;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t ctarank = cluster_ctarank();
  const uint32_t rank = ctarank & 1u;      // in the pair
  const uint32_t leader = ctarank & ~1u;   // the pair's rank 0
  const int n_stages = L::stages(g.tn);
  const int stage_bytes = L::stage_bytes(g.tn);
  uint8_t* stages = smem + L::kStageOffset;
  if (threadIdx.x == 0) {
    for (int s = 0; s < n_stages; ++s) {
      mbar_init(&full[s], 2);  // armed by rank 0's two producers with both CTAs' bytes
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&acc_full[a], 1);
      mbar_init(&acc_empty[a], 2 * kTileEpiWarps);  // every epilogue warp of both CTAs
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, L::kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // both CTAs' barriers initialised before any remote use
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  grid_dependents_launch();
  grid_dependency_wait();

  const int total = g.n_tb * g.n_nt;
  // SPLIT: one tile per cluster; else the pairs stride over the tiles
  const int unit0 = static_cast<int>(SPLIT ? blockIdx.x / (2u * static_cast<unsigned>(g.split)) : blockIdx.x >> 1);
  const int n_units = SPLIT ? total : static_cast<int>(gridDim.x >> 1);
  // stages of a tile along K (SPLIT: this pair's share), and accumulations they are cut into
  const int ns_all = (g.nk + kLinAtoms - 1) / kLinAtoms;
  const int s_first = SPLIT ? static_cast<int>(static_cast<long long>(ns_all) * (ctarank >> 1) / g.split) : 0;
  const int s_end = SPLIT ? static_cast<int>(static_cast<long long>(ns_all) * ((ctarank >> 1) + 1) / g.split) : ns_all;
  const int ns = s_end - s_first;
  const int kc_stages = !PROMOTE ? ns : SPLIT ? (ns + 1) / 2 : kPromoteAtoms / kLinAtoms;
  const int n_kc = PROMOTE ? (ns + kc_stages - 1) / kc_stages : 1;
  const int b_rows = g.tn / 2;  // weight rows in each CTA

  if (warp == 0 || warp == 2) {
    if (elect_one()) {
      const bool is_x = warp == 0;
      const CUtensorMap* tm = is_x ? &tmX : &tmW;
      const CUtensorMap* tail = is_x ? &tmXt : &tmWt;
      const uint64_t pol = policy_evict_last();  // both operands are read by several tiles
      const uint32_t full0 = mapa_shared(smem_u32(full), leader);
      const int atom_bytes = is_x ? L::kAtom : b_rows * kTileKBytes;
      const int off = is_x ? 0 : L::kABytes;
      int stage = 0;
      uint32_t phase = 0;
      uint32_t pending = 0, parity = 0;
      bool ok = true;
      for (int tile = unit0; tile < total && ok; tile += n_units) {
        int mt, nt;
        tile_coords(g, tile, mt, nt);
        const int row0 = is_x ? mt * 2 * kTileM + static_cast<int>(rank) * kTileM
                              : nt * g.tn + static_cast<int>(rank) * b_rows;
        for (int ks = s_first; ks < s_end; ++ks) {
          ok = mbar_wait(&empty[stage], phase ^ 1u, abort_flag);
          if (!ok) break;
          const int na = min(kLinAtoms, g.nk - ks * kLinAtoms);
          if (rank == 0) mbar_arrive_expect_tx(&full[stage], static_cast<uint32_t>(2 * na * atom_bytes));
          load_stage<KE, true>(stages + stage * stage_bytes + off, tm, tail, nullptr,
                               full0 + 8u * static_cast<uint32_t>(stage), ks, row0, atom_bytes, g, pol);
          pending |= 1u << stage;
          parity = (parity & ~(1u << stage)) | (phase << stage);
          if (++stage == n_stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (ok) {
        // The releases that no refill waited for: one may not reach this CTA's barrier after its end, where a kernel
        // that started early may have its own. (k_linear_split does not send them, 0.3 us better where a launch takes
        // 5; here that test in the MMA loop cost 2 % at 3532 x 5641 x 1408, and these waits pass during the epilogue.)
        for (int i = 0; i < n_stages && ok; ++i) {
          ok = mbar_wait(&empty[stage], phase ^ 1u, abort_flag);
          if (++stage == n_stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      } else {
        if (rank == 0) {
          for (int s = 0; s < n_stages; ++s)
            if ((pending >> s) & 1u) drain_wait(&full[s], (parity >> s) & 1u);
        } else if (pending) {
          // rank 1's copies complete on rank 0's barriers, which it cannot wait
          // on: give copies in flight a bounded 2 ms to land before unwinding
          const uint64_t t0 = globaltimer();
          while (globaltimer() - t0 < 2000000ull) __nanosleep(1000);
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0 && elect_one()) {
      const uint32_t idesc = FP8 ? idesc_e4m3(2 * kTileM, g.tn) : idesc_16bit(2 * kTileM, g.tn, g.f16);
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      int j = 0;  // accumulation counter: accumulator j % 2
      const uint16_t pair_mask = static_cast<uint16_t>(3u << leader);
      for (int tile = unit0; tile < total && ok; tile += n_units) {
        for (int kc = 0; kc < n_kc && ok; ++kc, ++j) {
          const int acc = j & 1;
          ok = mbar_wait(&acc_empty[acc], ((static_cast<uint32_t>(j) >> 1) & 1u) ^ 1u, abort_flag);
          if (!ok) break;
          tc_fence_after();
          const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * 256);
          const int s_lo = s_first + kc * kc_stages, s_hi = min(s_end, s_lo + kc_stages);
          for (int ks = s_lo; ks < s_hi; ++ks) {
            ok = mbar_wait(&full[stage], phase, abort_flag);
            if (!ok) break;
            tc_fence_after();
            const int na = min(kLinAtoms, g.nk - ks * kLinAtoms);
            const uint32_t a_addr = smem_u32(stages + stage * stage_bytes);
#pragma unroll
            for (int a = 0; a < kLinAtoms; ++a) {
              if (a < na) {
                const uint64_t adesc = sw128_kmajor_desc(a_addr + a * L::kAtom);
                const uint64_t bdesc = sw128_kmajor_desc(a_addr + L::kABytes + a * b_rows * kTileKBytes);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                  const uint32_t accum = (ks != s_lo || (a | kk) != 0) ? 1u : 0u;
                  if (FP8) umma_f8_pair(d_tmem, adesc + 2 * kk, bdesc + 2 * kk, idesc, accum);
                  else umma_f16_pair(d_tmem, adesc + 2 * kk, bdesc + 2 * kk, idesc, accum);
                }
              }
            }
            umma_commit_pair_multicast(&empty[stage], pair_mask);
            if (++stage == n_stages) {
              stage = 0;
              phase ^= 1u;
            }
          }
          if (ok) umma_commit_pair_multicast(&acc_full[acc], pair_mask);
        }
      }
      if (ok) {
        // the epilogue's last releases: rank 1's are remote arrivals that the relaxed cluster barrier does not order
        if (!SPLIT) {
          for (int acc = 0; acc < 2 && ok; ++acc) {
            const int uses = acc_uses(j, acc);
            if (uses > 0) ok = mbar_wait(&acc_empty[acc], last_release_parity(uses), abort_flag);
          }
        }
      } else {
        umma_commit_pair(mapa_shared(smem_u32(drain), leader));
        drain_wait(drain, 0);
      }
    }
    __syncwarp();
  } else if (SPLIT && warp >= 3) {
    // partial tile to shared memory: the stages are free once the last accumulation is complete
    const int q = warp & 3;
    const int r = 32 * q + lane;
    bool ok = true;
    for (int kc = 0; kc < n_kc && ok; ++kc) ok = mbar_wait(&acc_full[kc], 0, abort_flag);
    ok = __all_sync(0xffffffffu, ok);
    if (ok) {
      tc_fence_after();
      float4* part = reinterpret_cast<float4*>(stages);
      for (int c = (warp - 3) >> 2; c < g.tn / 32; c += 2) {
        const uint32_t at = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + static_cast<uint32_t>(32 * c);
        float v[32];
        tmem_ld32(at, v);
        tmem_wait_ld();
        if (PROMOTE && n_kc == 2) {
          float v2[32];
          tmem_ld32(at + 256, v2);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] += v2[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
          part[part_unit(r, 8 * c + i, g.tn)] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
      }
    }
  } else if (!SPLIT && warp >= 3) {
    const int ew = warp - 3;
    const int q = warp & 3;    // TMEM lane quarter
    const int half = ew >> 2;  // columns 32 c.. with c % 2 == half
    uint8_t* st = smem + ew * L::kWarpOut;
    const uint32_t acc_empty0 = mapa_shared(smem_u32(acc_empty), leader);
    const int chunks = g.tn / 32;
    int j = 0;
    bool ok = true;
    for (int tile = unit0; tile < total && ok; tile += n_units) {
      int mt, nt;
      tile_coords(g, tile, mt, nt);
      const int row0 = mt * 2 * kTileM + static_cast<int>(rank) * kTileM + 32 * q;
      const int t = row0 + lane;
      const float xs = g.x_scale && t < g.T ? g.x_scale[t] : 1.f;
      const uint32_t t_row = tmem_base + (static_cast<uint32_t>(32 * q) << 16);

      // weight scale, bias and residual of chunk c, fetched a chunk ahead
      float ws = 1.f, bias = 0.f;
      uint32_t res[16];
      auto fetch = [&](int c) {
        const int n0 = nt * g.tn + 32 * c;
        const bool in = c < chunks && row0 < g.T && n0 + lane < g.N;
        if (FP8) ws = in ? g.w_scale[static_cast<size_t>(n0 + lane) * g.w_scale_step] : 1.f;
        if (g.bias) bias = in ? load_typed(g.bias, g.bias_dt, n0 + lane) : 0.f;
        if (!PROMOTE && g.residual && c < chunks && row0 < g.T && n0 < g.N) fetch_residual<2, U>(g, res, row0, n0, lane);
      };
      auto finish = [&](float (&v)[32], int c) {
        const int n0 = nt * g.tn + 32 * c;
        const bool in = row0 < g.T && n0 < g.N;
        float* vec = reinterpret_cast<float*>(st);  // scales and bias to every lane, through the staging
        if (FP8) vec[lane] = ws;
        vec[32 + lane] = bias;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (FP8) {
            const float4 w = reinterpret_cast<const float4*>(vec)[i];
            v[4 * i] = v[4 * i] * xs * w.x;
            v[4 * i + 1] = v[4 * i + 1] * xs * w.y;
            v[4 * i + 2] = v[4 * i + 2] * xs * w.z;
            v[4 * i + 3] = v[4 * i + 3] * xs * w.w;
          }
          const float4 b = reinterpret_cast<const float4*>(vec)[8 + i];
          v[4 * i] += b.x;
          v[4 * i + 1] += b.y;
          v[4 * i + 2] += b.z;
          v[4 * i + 3] += b.w;
        }
        __syncwarp();
        if (!in) return;
        uint32_t r[16];
        if (PROMOTE) {
          if (g.residual) fetch_residual<4, U>(g, r, row0, n0, lane);
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) r[i] = res[i];
        }
        fetch(c + 2);
        apply_act<PROMOTE>(v, g.act);
        if (PROMOTE) tile_store_32<U>(g, st, v, r, row0, n0, lane);
        else if (g.out_dt == 0) tile_store_16<__nv_bfloat16, U>(g, st, v, r, row0, n0, lane);
        else tile_store_16<__half, U>(g, st, v, r, row0, n0, lane);
      };
      fetch(half);
      auto release = [&](int acc) {
        tc_fence_before();
        __syncwarp();
        // relaxed: the TMEM reads are complete, and the result stores of earlier chunks need not land first
        if (lane == 0) mbar_arrive_cluster_relaxed(acc_empty0 + 8u * static_cast<uint32_t>(acc));
      };

      if constexpr (PROMOTE) {
        float sum[kPromoteTn / 64][32];
        for (int kc = 0; kc < n_kc; ++kc, ++j) {
          const int acc = j & 1;
          ok = mbar_wait(&acc_full[acc], (static_cast<uint32_t>(j) >> 1) & 1u, abort_flag);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int i = 0; i < kPromoteTn / 64; ++i) {
            const int c = 2 * i + half;
            if (c < chunks) {
              float v[32];
              tmem_ld32(t_row + static_cast<uint32_t>(acc * 256 + 32 * c), v);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) sum[i][e] = kc == 0 ? v[e] : sum[i][e] + v[e];
            }
          }
          release(acc);
        }
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < kPromoteTn / 64; ++i)
          if (2 * i + half < chunks) finish(sum[i], 2 * i + half);
      } else {
        const int acc = j & 1;
        ok = mbar_wait(&acc_full[acc], (static_cast<uint32_t>(j) >> 1) & 1u, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        for (int c = half; c < chunks; c += 2) {
          float v[32];
          tmem_ld32(t_row + static_cast<uint32_t>(acc * 256 + 32 * c), v);
          tmem_wait_ld();
          if (c + 2 >= chunks) release(acc);
          finish(v, c);
        }
        ++j;
      }
    }
  }

  if constexpr (SPLIT) {
    cluster_sync_all();  // every partial tile is written
    if (warp >= 3) {
      int mt, nt;
      tile_coords(g, unit0, mt, nt);
      split_rows<PROMOTE>(g, smem_u32(stages), ctarank, mt, nt, warp - 3, lane);
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_relaxed();  // no CTA leaves while its peer's roles still wait on or signal its barriers
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, L::kTmemCols);
  }
}

}  // namespace moe
