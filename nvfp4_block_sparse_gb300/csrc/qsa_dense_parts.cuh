// qsa_dense_parts.cuh -- device code of the decode kernels of dense attention
// (qsa_dense.cu over NVFP4 pages, qsa_dense8.cu over 8-bit ones): asynchronous
// copies, and the join of a divided unit's records.
#pragma once

#include "qsa_dense.cuh"

namespace qsa {
namespace dense {

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a));
  return r;
}
// A sink's logit joins the denominator: new base and sum, and the factor of what was summed.
__device__ __forceinline__ void add_sink(float sink, float& m, float& l, float& f) {
  const float s2 = sink * kLog2e, nm = fmaxf(m, s2);
  f = exp2_approx(m - nm);
  l = l * f + exp2_approx(s2 - nm);
  m = nm;
}

// The records of a unit's parts (CTAs first..last) joined by a CTA of W warps, in the
// parts' order: W / vecs warps to a vector, each with every so-manieth part, then their
// sums in the warps' order.
// (kChkOut: the file's bounds-check code of an output row.)
template <int D, int W, int kChkOut>
__device__ __forceinline__ void join_parts(const Shape& sh, const Work& p, int b, int vec0, int vecs,
                                           int kvh, int first, int last, float* s_sum) {
  constexpr int E = D / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int parts = last - first + 1, ways = max(W / vecs, 1);
  const size_t rf = record_floats(sh.vt, D);
  auto record = [&](int i) {   // slot 1 of the first CTA, slot 0 of the others
    return p.records + ((size_t)(first + i) * 2 + (i == 0 ? 1 : 0)) * rf;
  };
  for (int c0 = 0; c0 < vecs; c0 += W) {
    const int c = c0 + warp % min(vecs, W), way = warp / min(vecs, W);
    const bool on = c < vecs && way < ways;
    float m = kNoBase, l = 0.f, acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    if (on) {
      for (int i = lane; i < parts; i += 32) m = fmaxf(m, __ldcg(record(i) + c));
#pragma unroll
      for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
#pragma unroll 4
      for (int i = way; i < parts; i += ways) {
        const float* rec = record(i);
        const float f = exp2_approx(__ldcg(rec + c) - m);
        l = fmaf(__ldcg(rec + sh.vt + c), f, l);
        const float4* src = reinterpret_cast<const float4*>(rec + 2 * sh.vt + (size_t)c * D) + lane * (E / 4);
#pragma unroll
        for (int e = 0; e < E / 4; ++e) {
          const float4 x = __ldcg(src + e);
          acc[4 * e] = fmaf(x.x, f, acc[4 * e]);
          acc[4 * e + 1] = fmaf(x.y, f, acc[4 * e + 1]);
          acc[4 * e + 2] = fmaf(x.z, f, acc[4 * e + 2]);
          acc[4 * e + 3] = fmaf(x.w, f, acc[4 * e + 3]);
        }
      }
    }
    if (ways > 1) {
      float* mine = s_sum + warp * (D + 4);
#pragma unroll
      for (int e = 0; e < E; ++e) mine[lane * E + e] = acc[e];
      if (lane == 0) mine[D] = l;
      __syncthreads();
      if (on && way == 0)
        for (int w = 1; w < ways; ++w) {
          const float* other = s_sum + (warp + w * min(vecs, W)) * (D + 4);
#pragma unroll
          for (int e = 0; e < E; ++e) acc[e] += other[lane * E + e];
          l += other[D];
        }
    }
    if (!on || way != 0) continue;
    const int j = row_of(sh, vec0 + c), head = kvh * sh.G + (vec0 + c) - j * sh.G;
    const size_t row = ((size_t)b * sh.g.R + j) * sh.g.Hq + head;
    if (!QSA_IN_BOUNDS(b < sh.g.B && j < sh.g.R && head < sh.g.Hq, kChkOut)) continue;
    float f = 1.f;
    if (p.sinks) add_sink(p.sinks[head], m, l, f);
    const float r = l == 0.f ? 0.f : f * p.v_scale / l;
    uint32_t w2[E / 2];
#pragma unroll
    for (int e = 0; e < E / 2; ++e) {
      const __nv_bfloat162 x = __floats2bfloat162_rn(acc[2 * e] * r, acc[2 * e + 1] * r);
      w2[e] = *reinterpret_cast<const uint32_t*>(&x);
    }
    if constexpr (E == 4)
      *reinterpret_cast<uint2*>(p.out + row * D + lane * E) = make_uint2(w2[0], w2[1]);
    else
      *reinterpret_cast<uint4*>(p.out + row * D + lane * E) = make_uint4(w2[0], w2[1], w2[2], w2[3]);
    if (lane == 0) p.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
  }
}

// A CTA's part of a unit done: the states of its warps (output fragments o, bases and sums) are
// joined over the ring in shared memory, whose copies have landed and been read, and the unit is
// written out, or, where it is divided, a record of the part; the last CTA to be done with the unit
// joins its records.  dim_of(gid, i): the first of the two neighbouring dims that rows gid and
// gid + 8 of output tile i stand for.  s_flag: a word of shared memory.
template <class C, int kChkOut, int kChkJoin, class DimOf>
__device__ __forceinline__ void finish_unit(const Shape& sh, const Work& p, const Span& span, const Cursor& cursor,
                                            const Seg& seg, uint8_t* smem, int* s_flag,
                                            float (&o)[C::DT][C::NT][4], float (&base)[C::NT][2],
                                            float (&sum)[C::NT][2], DimOf dim_of) {
  constexpr int D = C::D, NT = C::NT, W = C::W, DT = C::DT, kCols = C::kCols;
  const Geom& g = sh.g;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gid = lane >> 2, tig = lane & 3;
  const int b = seg.b, kvh = seg.kvh, vec0 = seg.vec0, vecs = seg.vecs;
  const bool begins = seg.begins, ends = seg.ends;
  // Fragment by fragment as the lanes hold them (no bank conflicts): thread (i, t, lane)
  // adds up the W warps' four values of two vectors and two dims.
  float* j_base = reinterpret_cast<float*>(smem);        // [W][kCols]
  float* j_sum = j_base + W * kCols;                     // [W][kCols]
  float4* j_o = reinterpret_cast<float4*>(j_sum + W * kCols);   // [W][DT][NT][32]
#pragma unroll
  for (int t = 0; t < NT; ++t) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float x = sum[t][e];
#pragma unroll
      for (int s2 = 4; s2 < 32; s2 <<= 1) x += __shfl_xor_sync(0xffffffffu, x, s2);
      if (gid == 0) {
        j_base[warp * kCols + 8 * t + 2 * tig + e] = base[t][e];
        j_sum[warp * kCols + 8 * t + 2 * tig + e] = x;
      }
    }
#pragma unroll
    for (int i = 0; i < DT; ++i)
      j_o[((warp * DT + i) * NT + t) * 32 + lane] =
          make_float4(o[i][t][0], o[i][t][1], o[i][t][2], o[i][t][3]);
  }
  __syncthreads();
  const bool whole = begins && ends;
  float* rec = p.records + ((size_t)blockIdx.x * 2 + (begins ? 1 : 0)) * record_floats(sh.vt, D);
  for (int x = tid; x < DT * NT * 32; x += C::kThreads) {
    const int i = x / (NT * 32), t = (x / 32) % NT;
    float acc[4] = {0.f, 0.f, 0.f, 0.f}, l[2] = {0.f, 0.f}, m[2] = {kNoBase, kNoBase};
    const int c0 = 8 * t + 2 * tig;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float2 bs = *reinterpret_cast<const float2*>(j_base + w * kCols + c0);
      m[0] = fmaxf(m[0], bs.x);
      m[1] = fmaxf(m[1], bs.y);
    }
#pragma unroll 4
    for (int w = 0; w < W; ++w) {
      const float4 v = j_o[((w * DT + i) * NT + t) * 32 + lane];
      const float2 ls = *reinterpret_cast<const float2*>(j_sum + w * kCols + c0);
      const float2 bs = *reinterpret_cast<const float2*>(j_base + w * kCols + c0);
      const float2 f = make_float2(exp2_approx(bs.x - m[0]), exp2_approx(bs.y - m[1]));
      acc[0] = fmaf(v.x, f.x, acc[0]);
      acc[1] = fmaf(v.y, f.y, acc[1]);
      acc[2] = fmaf(v.z, f.x, acc[2]);
      acc[3] = fmaf(v.w, f.y, acc[3]);
      l[0] = fmaf(ls.x, f.x, l[0]);
      l[1] = fmaf(ls.y, f.y, l[1]);
    }
    const int d = dim_of(gid, i);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int c = c0 + e;
      if (c >= vecs) continue;
      if (whole) {
        const int j = row_of(sh, vec0 + c), head = kvh * sh.G + (vec0 + c) - j * sh.G;
        const size_t row = ((size_t)b * g.R + j) * g.Hq + head;
        if (!QSA_IN_BOUNDS(b < g.B && j < g.R && head < g.Hq, kChkOut)) continue;
        float f = 1.f;
        if (p.sinks) add_sink(p.sinks[head], m[e], l[e], f);
        const float r = l[e] == 0.f ? 0.f : f * p.v_scale / l[e];
        *reinterpret_cast<__nv_bfloat162*>(p.out + row * D + d) =
            __floats2bfloat162_rn(acc[e] * r, acc[2 + e] * r);
        if (d == 0) p.lse[row] = l[e] == 0.f ? -INFINITY : (m[e] + log2f(l[e])) * kLn2;
      } else {
        if (d == 0) {
          rec[c] = m[e];
          rec[sh.vt + c] = l[e];
        }
        *reinterpret_cast<float2*>(rec + 2 * sh.vt + (size_t)c * D + d) = make_float2(acc[e], acc[2 + e]);
      }
    }
  }

  // ---- a divided unit: the last CTA to be done with it joins its records -------------
  if (!whole) {
    const int first = cursor.first_cta(sh, span.share), last = cursor.last_cta(sh, seg, span.share);
    __threadfence();
    __syncthreads();
    if (tid == 0 && !QSA_IN_BOUNDS(first >= 0 && first < last && last < sh.ctas, kChkJoin)) {
      *s_flag = 0;
    } else if (tid == 0) {
      const int before = atomicAdd(&p.tickets[last], 1);
      *s_flag = before == last - first;
      if (before == last - first) p.tickets[last] = 0;
    }
    __syncthreads();
    if (*s_flag) {
      __threadfence();
      join_parts<D, W, kChkOut>(sh, p, b, vec0, vecs, kvh, first, last, reinterpret_cast<float*>(smem));
    }
  }
}

}  // namespace dense
}  // namespace qsa
