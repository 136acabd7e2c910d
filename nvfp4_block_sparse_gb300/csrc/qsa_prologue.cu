// qsa_prologue.cu -- what a step does to its new rows before attention: the
// rotation rows of its positions, norms of the query and key heads with the
// rotation in the same pass, the append of rotated keys and of values to the
// NVFP4 pages, and cache rows read back.
//
// TensorRT-LLM PR #20276 ("Qwen3.8-Flash-Next NVFP4 target"), Performance
// (what runs on the fast paths): the attention prologue does QK norm and rope,
// the index store and the NVFP4 store; Known limitations: context rows read
// the pages dequantised to bf16.
//
// Arithmetic.  Everything between the bf16 inputs and the one rounding at the
// end is an IEEE fp32 operation in the order that the header states (products
// and sums kept apart, a pairwise sum of squares, an IEEE square root and
// division), so that the bytes in the cache are a function of the inputs
// alone, equal on every machine, and the fused append gives the bytes of its
// two parts called one after the other.
#include "qsa_common.cuh"

namespace qsa {
namespace {

// Bounds-check codes (reported by bounds-checked builds only).
[[maybe_unused]] constexpr int kChkRow = 0x801;    // append: pool row out of range
[[maybe_unused]] constexpr int kChkLoad = 0x802;   // read-back: pool row out of range

// ---------------------------------------------------------------------------
// Rotation rows.  A frequency is a 64-bit fraction of a turn, so pos * turns
// modulo 2^64 is the angle as a fraction of a turn whatever the position; its
// upper 32 bits, signed, lie in [-1/2, 1/2) turn and sincospif takes them
// without a further reduction.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256)
rope_rows_kernel(int R, long long T, const __grid_constant__ qsa_rope_t rope,
                 const int32_t* __restrict__ seqlens, const int32_t* __restrict__ positions,
                 float2* __restrict__ cs) {
  const int pairs = rope.rotary_dim >> 1;
  pdl_wait();
  pdl_trigger();
  const unsigned long long turns = rope.turns[threadIdx.x];
  for (long long r = (long long)blockIdx.x * blockDim.y + threadIdx.y; r < T;
       r += (long long)gridDim.x * blockDim.y) {
    const long long pos = positions ? positions[r]
                                    : (long long)seqlens[r / R] - R + (int)(r % R);
    const unsigned long long phase = (unsigned long long)pos * turns;
    const float turn = (float)(int)(phase >> 32) * 0x1p-31f;   // half turns
    float s, c;
    sincospif(turn, &s, &c);
    cs[r * pairs + threadIdx.x] = make_float2(c * rope.amplitude, s * rope.amplitude);
  }
}

// ---------------------------------------------------------------------------
// Norms, rotation, append.
//
// A head of D elements belongs to D/8 lanes, eight elements (16 bytes) each: a
// warp holds two heads at D = 128, one at D = 256.  A warp takes STEPS times the
// heads it holds of one row, all requested before the first is used, and keeps
// the row's cos and sin in registers meanwhile.  The pairs of the half layout meet by a
// shuffle over rotary_dim / 16 lanes (rotary_dim is a multiple of 16, so a
// lane's eight elements have one partner lane); interleaved pairs are in the lane.
// ---------------------------------------------------------------------------
constexpr int kWarps = 8;

struct KernelArgs {
  Geom g;
  NormRope nr;
  PrologueArgs a;
  int groups;      // warps per row
  int total;       // heads per row: query, key and (append) value heads
};

__device__ __forceinline__ void unpack8(const uint4& r, float (&x)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int D, bool kAppend, bool kInter, int STEPS>
__global__ void __launch_bounds__(kWarps * 32)
prologue_kernel(const __grid_constant__ KernelArgs p) {
  constexpr int LPV = D / 8;        // lanes per head
  constexpr int VPW = 32 / LPV;     // heads that a warp holds
  const Geom& g = p.g;
  const PrologueArgs& a = p.a;
  const int lane = threadIdx.x & 31;
  const int l = lane % LPV, e0 = 8 * l;   // the lane's first element
  const uint32_t item = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const uint32_t T = (uint32_t)g.B * (uint32_t)g.R;
  pdl_wait();
  pdl_trigger();
  const uint32_t r = item / (uint32_t)p.groups;   // (2^24 rows of at most 2^7 warps)
  if (r >= T) return;
  const int v0 = (int)(item - r * (uint32_t)p.groups) * (VPW * STEPS);
  const int v1 = min(v0 + VPW * STEPS, p.total);
  const int hq = a.q ? g.Hq : 0;

  // all of the warp's heads are requested before anything waits for one
  uint4 raws[STEPS];
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    const int hv = v0 + i * VPW + lane / LPV;
    raws[i] = make_uint4(0u, 0u, 0u, 0u);
    if (hv < v1) {
      const __nv_bfloat16* src = hv < hq           ? a.q + r * a.q_stride + hv * D
                                 : hv < hq + g.Hkv ? a.k + r * a.k_stride + (hv - hq) * D
                                                   : a.v + r * a.v_stride + (hv - hq - g.Hkv) * D;
      raws[i] = *reinterpret_cast<const uint4*>(src + e0);
    }
  }

  // the lane's cos and sin: o = y c + partner s, with the sign of the first
  // half's sine in s
  const int rot = p.nr.rot, h = rot >> 1;
  const bool turned = e0 < rot;
  int partner = lane;
  float c[8], s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) { c[i] = 1.f; s[i] = 0.f; }
  if (turned && v0 < hq + g.Hkv) {
    const float2* row = reinterpret_cast<const float2*>(a.cs) + (size_t)r * h;
    if (kInter) {
      const float4* row4 = reinterpret_cast<const float4*>(row + (e0 >> 1));
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 t = __ldg(row4 + i);
        c[4 * i] = c[4 * i + 1] = t.x;
        s[4 * i] = -t.y;
        s[4 * i + 1] = t.y;
        c[4 * i + 2] = c[4 * i + 3] = t.z;
        s[4 * i + 2] = -t.w;
        s[4 * i + 3] = t.w;
      }
    } else {
      const bool first = e0 < h;
      partner = first ? lane + h / 8 : lane - h / 8;
      const float4* row4 = reinterpret_cast<const float4*>(row + (first ? e0 : e0 - h));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 t = __ldg(row4 + i);
        c[2 * i] = t.x;
        c[2 * i + 1] = t.z;
        s[2 * i] = first ? -t.y : t.y;
        s[2 * i + 1] = first ? -t.w : t.w;
      }
    }
  }

  // the row's slot in the cache
  size_t page_row = 0;
  int slot = 0;
  bool has_slot = false;
  if (kAppend && v1 > hq) {
    const uint32_t b = r / (uint32_t)g.R;
    const long long pos = (long long)a.seqlens[b] - g.R + (int)(r - b * (uint32_t)g.R);
    if (pos >= 0 && pos < (long long)g.MB * g.P) {
      const int at = (int)pos, beta = at / g.P;
      const int page = a.page_table[(size_t)b * g.MB + beta];
      slot = at - beta * g.P;
      has_slot = page >= 0 && page < g.NP;
      page_row = (size_t)(has_slot ? page : 0);
    }
    // the index key, by the row's last warp: 16 lanes x 4 B
    if (v1 == p.total && has_slot && lane < kIndexDim / 4) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(a.ik + (size_t)r * kIndexDim + 4 * lane);
      *reinterpret_cast<uint32_t*>(a.ik_pool + (page_row * g.P + slot) * kIndexDim + 4 * lane) = w;
    }
  }

  // Sums of squares, neighbours first: eight in the lane, then lanes 1, 2, 4, ...
  // apart.  Four steps' sums are folded into one another on the way (a lane passes on
  // the sums it does not keep), so that lane i ends with that of step i mod 4, and one
  // square root and division serve all four.
  float rms[STEPS];
  if (v0 < hq + g.Hkv && (a.q_weight || a.k_weight)) {
    float ss[STEPS];
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      float x[8];
      unpack8(raws[i], x);
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = __fmul_rn(x[k], x[k]);
#pragma unroll
      for (int n = 4; n; n >>= 1)
#pragma unroll
        for (int k = 0; k < n; ++k) x[k] = __fadd_rn(x[2 * k], x[2 * k + 1]);
      ss[i] = x[0];
    }
    float sum;
    if constexpr (STEPS == 4) {
      const bool odd = lane & 1, upper = lane & 2;
      const float k01 = odd ? ss[1] : ss[0], g01 = odd ? ss[0] : ss[1];
      const float k23 = odd ? ss[3] : ss[2], g23 = odd ? ss[2] : ss[3];
      const float s01 = __fadd_rn(k01, __shfl_xor_sync(0xffffffffu, g01, 1));
      const float s23 = __fadd_rn(k23, __shfl_xor_sync(0xffffffffu, g23, 1));
      sum = __fadd_rn(upper ? s23 : s01, __shfl_xor_sync(0xffffffffu, upper ? s01 : s23, 2));
    } else {
      sum = ss[0];
    }
#pragma unroll
    for (int k = STEPS == 4 ? 4 : 1; k < LPV; k <<= 1)
      sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, k));
    const float inv = __fdiv_rn(1.f, __fsqrt_rn(__fadd_rn(sum * (1.f / D), p.nr.eps)));
#pragma unroll
    for (int i = 0; i < STEPS; ++i)
      rms[i] = STEPS == 4 ? __shfl_sync(0xffffffffu, inv, (lane & ~(LPV - 1)) + i) : inv;
  }

  float w[8];
  int w_kind = -1;
#pragma unroll
  for (int step = 0; step < STEPS; ++step) {
    if (STEPS > 1 && v0 + step * VPW >= v1) break;
    // warp-wide shuffles below: a lane without a head takes part with zeros
    const int hv = v0 + step * VPW + lane / LPV;
    const bool real = hv < v1;
    const int kind = hv < hq ? 0 : hv < hq + g.Hkv ? 1 : 2;   // query, key, value
    const int head = kind == 0 ? hv : kind == 1 ? hv - hq : hv - hq - g.Hkv;
    uint4 raw = raws[step];
    float x[8];
    unpack8(raw, x);
    if (v0 + step * VPW < hq + g.Hkv) {     // a query or key among the warp's heads
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = x[i];
      const __nv_bfloat16* weight = kind == 0 ? a.q_weight : a.k_weight;
      if (weight && kind < 2) {
        if (kind != w_kind) {
          w_kind = kind;
          unpack8(__ldg(reinterpret_cast<const uint4*>(weight + e0)), w);
          if (p.nr.plus_one) {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = __fadd_rn(1.f, w[i]);
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = __fmul_rn(__fmul_rn(x[i], rms[step]), w[i]);
      }
      if (rot) {
        if (kInter) {
          if (turned) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float u = y[2 * i], t = y[2 * i + 1];
              y[2 * i] = __fadd_rn(__fmul_rn(u, c[2 * i]), __fmul_rn(t, s[2 * i]));
              y[2 * i + 1] = __fadd_rn(__fmul_rn(t, c[2 * i + 1]), __fmul_rn(u, s[2 * i + 1]));
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float t = __shfl_sync(0xffffffffu, y[i], partner);
            if (turned) y[i] = __fadd_rn(__fmul_rn(y[i], c[i]), __fmul_rn(t, s[i]));
          }
        }
      }
      if (kind < 2) {
        raw = pack8(y);
        if (kAppend) unpack8(raw, x);
        if (real && kind == 0)
          *reinterpret_cast<uint4*>(a.q_out + ((size_t)r * g.Hq + head) * D + e0) = raw;
        if (!kAppend && real && kind == 1)
          *reinterpret_cast<uint4*>(a.k_out + ((size_t)r * g.Hkv + head) * D + e0) = raw;
      }
    }
    if (!kAppend || min(v0 + (step + 1) * VPW, v1) <= hq) continue;   // (queries alone)

    // keys and values: blocks of 16 (two lanes) to e2m1 codes and an e4m3 scale,
    // as the token store quantises them
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    if (!real || kind == 0 || !has_slot) continue;
    const float scale = kind == 2 ? a.v_scale : a.k_scale;
    const uint32_t sf = f32_to_e4m3(__fdiv_rn(__fdiv_rn(m, 6.0f), scale));
    const float den = __fmul_rn(e4m3_to_f32(sf), scale);
    uint32_t codes = 0;
    if (den != 0.f) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        codes |= canon_zero(f32x2_to_e2m1x2(__fdiv_rn(x[2 * i], den),
                                            __fdiv_rn(x[2 * i + 1], den))) << (8 * i);
    }
    const size_t row = (page_row * g.Hkv + head) * g.P + slot;
    if (!QSA_IN_BOUNDS(row < (size_t)g.NP * g.Hkv * g.P, kChkRow)) continue;
    uint8_t* pool = kind == 2 ? a.v_pool : a.k_pool;
    uint8_t* sfp = kind == 2 ? a.v_sf : a.k_sf;
    *reinterpret_cast<uint32_t*>(pool + row * (D / 2) + 4 * l) = codes;
    if (!(l & 1)) sfp[row * (D / 16) + (l >> 1)] = (uint8_t)sf;
  }
}

// ---------------------------------------------------------------------------
// Cache rows read back: eight elements (4 code bytes, one scale) per lane.
// ---------------------------------------------------------------------------
template <int D>
__global__ void __launch_bounds__(kWarps * 32)
load_tokens_kernel(Geom g, const int32_t* __restrict__ page_table,
                   const int32_t* __restrict__ seqlens, const uint8_t* __restrict__ k_pool,
                   const uint8_t* __restrict__ k_sf, const uint8_t* __restrict__ v_pool,
                   const uint8_t* __restrict__ v_sf, float k_scale, float v_scale,
                   __nv_bfloat16* __restrict__ k_out, __nv_bfloat16* __restrict__ v_out) {
  constexpr int LPV = D / 8;
  const long long item = (long long)blockIdx.x * (kWarps * 32 / LPV) + threadIdx.x / LPV;
  const int l = threadIdx.x % LPV;
  const long long rows = (long long)g.B * g.R;
  pdl_wait();
  pdl_trigger();
  if (item >= rows * g.Hkv * 2) return;
  const int head2 = (int)(item % (2 * g.Hkv));
  const bool is_v = head2 >= g.Hkv;
  const int head = is_v ? head2 - g.Hkv : head2;
  const long long r = item / (2 * g.Hkv);
  const int b = (int)(r / g.R), j = (int)(r % g.R);
  const long long pos = (long long)seqlens[b] - g.R + j;
  if (pos < 0 || pos >= (long long)g.MB * g.P) return;
  const int page = page_table[(size_t)b * g.MB + (int)(pos / g.P)];
  if (page < 0 || page >= g.NP) return;
  const size_t row = ((size_t)page * g.Hkv + head) * g.P + (int)(pos % g.P);
  if (!QSA_IN_BOUNDS(row < (size_t)g.NP * g.Hkv * g.P, kChkLoad)) return;
  const uint32_t w =
      *reinterpret_cast<const uint32_t*>((is_v ? v_pool : k_pool) + row * (D / 2) + 4 * l);
  const float sf = e4m3_to_f32((is_v ? v_sf : k_sf)[row * (D / 16) + (l >> 1)]);
  const float scale = is_v ? v_scale : k_scale;
  float x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t h2 = e2m1x2_to_f16x2((w >> (8 * i)) & 0xFFu);
    // code * block scale is exact in fp32; the tensor scale rounds once
    x[2 * i] = __fmul_rn(__half2float(__ushort_as_half((unsigned short)(h2 & 0xFFFFu))) * sf, scale);
    x[2 * i + 1] = __fmul_rn(__half2float(__ushort_as_half((unsigned short)(h2 >> 16))) * sf, scale);
  }
  *reinterpret_cast<uint4*>((is_v ? v_out : k_out) + ((size_t)r * g.Hkv + head) * D + 8 * l) = pack8(x);
}

template <class... Ex, class... Ac>
cudaError_t launch(void (*kern)(Ex...), dim3 grid, dim3 block, bool pdl, cudaStream_t stream,
                   Ac&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<Ac&&>(args)...);
}

}  // namespace

cudaError_t launch_rope_rows(const Geom& g, const qsa_rope_t& rope, const int32_t* seqlens,
                             const int32_t* positions, float* cs, bool pdl, cudaStream_t stream) {
  const int pairs = rope.rotary_dim / 2;
  const dim3 block(pairs, 256 / pairs);
  const long long T = (long long)g.B * g.R;
  const long long ctas = (T + block.y - 1) / block.y;
  return launch(rope_rows_kernel, dim3((unsigned)(ctas < 2432 ? ctas : 2432)), block, pdl, stream,
                g.R, T, rope, seqlens, positions, reinterpret_cast<float2*>(cs));
}

cudaError_t launch_prologue(const Geom& g, const NormRope& nr, const PrologueArgs& a, bool pdl,
                            cudaStream_t stream) {
  const bool append = a.v != nullptr;
  KernelArgs p;
  p.g = g;
  p.nr = nr;
  p.a = a;
  p.total = (a.q ? g.Hq : 0) + (append ? 2 : 1) * g.Hkv;
  const int vpw = g.D == 128 ? 2 : 1;
  const long long T = (long long)g.B * g.R;
  // Few rows: a warp per step of heads, for the shortest chain; many rows: four
  // steps per warp share the row's cos and sin.
  const int steps = T * p.total / vpw > 152 * 64 ? 4 : 1;
  p.groups = (p.total + vpw * steps - 1) / (vpw * steps);
  const long long items = T * p.groups;
  auto launch_it = [&]<int D, bool kAppend, bool kInter>() {
    auto* kern = steps == 4 ? prologue_kernel<D, kAppend, kInter, 4> : prologue_kernel<D, kAppend, kInter, 1>;
    return launch(kern, dim3((unsigned)((items + kWarps - 1) / kWarps)), dim3(kWarps * 32), pdl,
                  stream, p);
  };
  auto of_dim = [&]<int D>() {
    if (append)
      return nr.interleaved ? launch_it.template operator()<D, true, true>()
                            : launch_it.template operator()<D, true, false>();
    return nr.interleaved ? launch_it.template operator()<D, false, true>()
                          : launch_it.template operator()<D, false, false>();
  };
  return g.D == 256 ? of_dim.template operator()<256>() : of_dim.template operator()<128>();
}

cudaError_t launch_load_tokens(const Geom& g, const int32_t* page_table, const int32_t* seqlens,
                               const uint8_t* k_pool, const uint8_t* k_sf, const uint8_t* v_pool,
                               const uint8_t* v_sf, float k_scale, float v_scale, void* k_out,
                               void* v_out, bool pdl, cudaStream_t stream) {
  const int per = kWarps * 32 / (g.D / 8);
  const long long items = (long long)g.B * g.R * g.Hkv * 2;
  auto* kern = g.D == 256 ? load_tokens_kernel<256> : load_tokens_kernel<128>;
  return launch(kern, dim3((unsigned)((items + per - 1) / per)), dim3(kWarps * 32), pdl, stream, g,
                page_table, seqlens, k_pool, k_sf, v_pool, v_sf, k_scale, v_scale,
                reinterpret_cast<__nv_bfloat16*>(k_out), reinterpret_cast<__nv_bfloat16*>(v_out));
}

}  // namespace qsa

QSA_BOUNDS_READER(bounds_word_prologue)
