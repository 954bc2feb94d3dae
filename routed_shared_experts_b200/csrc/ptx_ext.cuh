// ptx_ext.cuh - further PTX wrappers: thread election, programmatic launch,
// relaxed cluster synchronisation, wider TMEM loads, multicast commits.
#pragma once
#include "ptx.cuh"

namespace moe {

// Routing id of a padding row of a batch: the sort drops its slots without an
// error, so that no expert works on them.
constexpr int32_t kNoExpert = INT32_MIN;

// True in one lane of a converged warp. The compiler knows a region under this
// predicate to be run by a single thread and keeps tensor-core descriptors and
// copy operands in uniform registers there; under `lane == 0` it moves them for
// every instruction (measured for a stage of eight MMAs and a commit, N = 16:
// 763 clocks under `lane == 0`, 403 under this).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred P;\n\t"
      "elect.sync _|P, 0xffffffff;\n\t"
      "selp.b32 %0, 1, 0, P;\n\t}\n"
      : "=r"(p));
  return p != 0;
}

// Programmatic launch of dependents: the first call lets the next kernel of the
// stream start once every CTA of this one has started, the second waits until
// the kernels before this one have completed and their writes are visible. A
// kernel launched with launch_early() (host) calls both before its first access
// to global memory, so only what comes before them - the launch itself, barriers,
// TMEM - overlaps its predecessor. Such a kernel loads its operands with plain
// loads: the read-only path (ld.global.nc) is defined for memory that nothing
// writes while the kernel runs, and the predecessor still does.
__device__ __forceinline__ void grid_dependents_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// A plain load that stays where it is written; the compiler is free to move others
// down to where their value is used.
__device__ __forceinline__ float ld_global_here(const float* p) {
  float v;
  asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
}

// 32 lanes x 32 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// mbar_arrive_cluster without ordering this thread's memory accesses: the release
// at cluster scope waits for every global store issued before it to reach L2.
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// Cluster barrier that orders nothing: for the end of a kernel, where a CTA
// only has to outlive its peers' accesses to its shared memory.
__device__ __forceinline__ void cluster_sync_relaxed() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// umma_commit_pair on the barrier at this shared::cta offset in every CTA of
// `mask` (bit = rank in the cluster).
__device__ __forceinline__ void umma_commit_pair_multicast(uint64_t* bar, uint16_t mask) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"(mask)
      : "memory");
}

}  // namespace moe
