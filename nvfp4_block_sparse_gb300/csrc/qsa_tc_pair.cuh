// qsa_tc_pair.cuh -- what the tensor-core kernels of dense and prompt attention share beyond
// qsa_tc.cuh: sleeping bounded waits, MMAs and commits of one CTA or of a pair, wide
// tensor-memory loads, packed fp32 arithmetic, register splits.
#pragma once

#include "qsa_tc.cuh"

namespace qsa {
namespace tc {

// 32 columns of this thread's lane.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// Two fp32 multiply-adds / additions at once.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mov.b64 z, {%6, %7};\n\tfma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// The sum of a long row's weights, joined chunk by chunk with what each addition's rounding loses (Kahan,
// 1965): next to 2^24 others of its size a weight would vanish, and of weights that are alike all
// roundings go one way (131072 tokens of one row in plain sums: lse off by 1.5e-3).  A chunk's own
// weights are added up first, so this is four packed operations in 128 tokens, for the even tokens and for the
// odd ones (one sum of both, which the next chunk waits for: a prompt of 8192 tokens 311 -> 320 us; so 311).
struct RowSum {
  float2 sum = make_float2(0.f, 0.f), lost = make_float2(0.f, 0.f);
  __device__ __forceinline__ void add(float2 part) {
    const float2 minus = make_float2(-1.f, -1.f), y = add2(part, lost), t = add2(sum, y);
    lost = fma2(fma2(sum, minus, t), minus, y);          // y - (t - sum)
    sum = t;
  }
  __device__ __forceinline__ void scale(float f) {
    sum.x *= f;
    sum.y *= f;
    lost.x *= f;
    lost.y *= f;
  }
  __device__ __forceinline__ float total() const { return sum.x + sum.y; }
};

// ---- rows of neighbouring lanes ------------------------------------------------
// Four lanes' rows of four 16-byte pieces transposed: lane j then has piece j of each of the four rows,
// so that a store writes runs of 64 bytes.
__device__ __forceinline__ void transpose4(uint32_t (&w)[16], int lane) {
  const bool odd = lane & 1, upper = lane & 2;
#pragma unroll
  for (int x = 0; x < 4; ++x) {
#pragma unroll
    for (int c = 0; c < 4; c += 2) {
      const uint32_t p = w[4 * c + x], q = w[4 * c + 4 + x];
      const uint32_t g = __shfl_xor_sync(0xffffffffu, odd ? p : q, 1);
      w[4 * c + x] = odd ? g : p;
      w[4 * c + 4 + x] = odd ? q : g;
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const uint32_t p = w[4 * c + x], q = w[4 * c + 8 + x];
      const uint32_t g = __shfl_xor_sync(0xffffffffu, upper ? p : q, 2);
      w[4 * c + x] = upper ? g : p;
      w[4 * c + 8 + x] = upper ? q : g;
    }
  }
}

// ---- barriers across the pair ------------------------------------------------
// One wait of at most about 20 us during which the thread sleeps in hardware.
__device__ __forceinline__ bool sleep_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(20000u)
      : "memory");
  return ok != 0;
}

// A warp's bounded wait: true when it gave up, in every lane.  It sleeps: a dozen
// warps polling (and reading the clock) slowed everything else on the SM down several times.
__device__ __forceinline__ bool gave_up(uint64_t* bar, uint32_t parity) {
  bool ok = sleep_wait(bar, parity & 1);
  if (!ok) {
    const unsigned long long t0 = now_ns();
    while (!(ok = sleep_wait(bar, parity & 1)) && now_ns() - t0 <= kWaitNs) {
    }
  }
  return __any_sync(0xffffffffu, !ok);
}

// The same for a barrier of each lane's own, where it has one.
__device__ __forceinline__ bool lanes_gave_up(uint64_t* bar, uint32_t parity, bool mine) {
  bool ok = !mine || sleep_wait(bar, parity & 1);
  if (!ok) {
    const unsigned long long t0 = now_ns();
    while (!(ok = sleep_wait(bar, parity & 1)) && now_ns() - t0 <= kWaitNs) {
    }
  }
  return __any_sync(0xffffffffu, !ok);
}

// One arrival of the warp at the first CTA's barrier.
template <int CG>
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) {
    if constexpr (CG == 1)
      ws_arrive(bar);
    else
      asm volatile(
          "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, 0;\n\t"
          "mbarrier.arrive.shared::cluster.b64 _, [a];\n\t}" ::"r"(smem_u32(bar))
          : "memory");
  }
}

// ---- MMAs by one lane of a converged warp ---------------------------------------
// The lane is elected once (`one` is 1 in it): the warp stays converged, so that the
// descriptors stay in uniform registers, and an MMA costs no election of its own (two
// context chunks 737 -> 673 us).
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(r));
  return r;
}
template <int CG>
__device__ __forceinline__ void mma_ss(uint32_t one, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  if constexpr (CG == 1)
    asm volatile(
        "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 e, %5, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(one));
  else
    asm volatile(
        "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 e, %5, 0;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(one));
}
template <int CG>
__device__ __forceinline__ void mma_ts(uint32_t one, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  if constexpr (CG == 1)
    asm volatile(
        "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 e, %5, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(one));
  else
    asm volatile(
        "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 e, %5, 0;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(one));
}
template <int CG>
__device__ __forceinline__ void commit(uint32_t one, uint64_t* bar) {
  if constexpr (CG == 1)
    asm volatile(
        "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %1, 0;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
            smem_u32(bar)), "r"(one)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %2, 0;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster"
        ".b64 [%0], %1;\n\t}" ::"r"(smem_u32(bar)), "h"((uint16_t)3), "r"(one)
        : "memory");
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

}  // namespace tc
}  // namespace qsa
