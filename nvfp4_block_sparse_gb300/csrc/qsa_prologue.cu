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
// modulo 2^64 is the angle as a fraction of a turn whatever the position, and
// sincospif takes it without a further reduction.  Errors: its one unit in the last place
// (6e-8), the correction's and the amplitude's roundings (3e-8, 6e-8 amplitude), the bits
// below 2^-32 turn (1e-9).  4 x 4096 rows of 32 pairs (4.2 MB): 5.1 us, bound by the
// lanes' reads of their frequencies from the parameters, which are served an address at a time
// (that unit is 84 % busy; instructions would issue in 2.4 us); 192 rows of 64 pairs: 1.5 us,
// a launch.
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
    // The upper 32 bits, signed, lie in [-1/2, 1/2) turn.  fp32 holds 24 of them; the others turn
    // sine and cosine by less than 1e-7, to first order.
    const int bits = (int)(phase >> 32);
    const float top = (float)bits;
    const float rest = (float)(bits - __float2int_rn(top)) * (3.14159265f * 0x1p-31f);
    float s, c;
    sincospif(top * 0x1p-31f, &s, &c);
    cs[r * pairs + threadIdx.x] = make_float2(fmaf(-s, rest, c) * rope.amplitude,
                                              fmaf(c, rest, s) * rope.amplitude);
  }
}

// ---------------------------------------------------------------------------
// Norms, rotation, append.
//
// A head of D elements belongs to D/8 lanes, eight elements (16 bytes) each: a
// warp holds two heads at D = 128, one at D = 256.  A warp's turn is STEPS times
// the heads it holds of one row's queries, or of its keys and, in the append, its values
// behind them (the few of both share a turn): all requested before the first is used, and with many rows the next turn's before this
// one's are worked on.  The row's cos and sin stay in registers meanwhile, and the
// arithmetic is on packed pairs.  The pairs of the half layout meet by a
// shuffle over rotary_dim / 16 lanes (rotary_dim is a multiple of 16, so a
// lane's eight elements have one partner lane); interleaved pairs are in the lane.
//
// Measured (GB300): norms and rotation of 8192 rows of 24 + 2 heads of 256 (220 MB) 39.8 us,
// 5.5 TB/s (0.83 of the measured copy rate), instructions issued in 61 % of the cycles: about
// 100 per head and warp.  The append of 8188 such rows with their values (223 MB) 47.8 us:
// its keys and values take four times the instructions of a query; see the quantiser below
// for what its divisions cost.  Steps (8192 rows): a turn per kind 77 us, next turn requested
// ahead 63.5, four square roots as one 51.7, packed arithmetic 42.
// ---------------------------------------------------------------------------
constexpr int kWarps = 4;

struct KernelArgs {
  Geom g;
  NormRope nr;
  PrologueArgs a;
  int turns_q, turns;            // turns per row: queries, all
  float k_inv6, v_inv6;          // 1 / (6 scale), or 0 where that is far from 1
};

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// y c + t s, each operation rounded.  Not by packed pairs: the assembler fuses a packed
// product and sum, which rounds once (seen as one flipped bf16 result in 10^5).  (The
// squares may be: products of bf16 values are exact.)
__device__ __forceinline__ float2 turn2(float2 y, float2 c, float2 t, float2 s) {
  return make_float2(__fadd_rn(__fmul_rn(y.x, c.x), __fmul_rn(t.x, s.x)),
                     __fadd_rn(__fmul_rn(y.y, c.y), __fmul_rn(t.y, s.y)));
}

__device__ __forceinline__ void unpack8(const uint4& r, float2 (&x)[4]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}

__device__ __forceinline__ uint4 pack8(const float2 (&x)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(x[i].x, x[i].y);
    w[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// A block of 16 values (this lane has eight, its neighbour the rest), of largest
// magnitude m, to codes and scale as the token store's divisions give them:
//   sf = e4m3((m / 6) / scale),  codes = e2m1(x / (e4m3(sf) scale)).
// Ten IEEE divisions per lane were most of the append's instructions.  A product
// with a reciprocal is within 2^-21 of the quotient; where 2^-20 to either side rounds
// to the same code, rounding being monotonic, so does the quotient.  Otherwise (about
// one block in 10^4), or where the scale is so small or large that the reciprocal is not
// a normal number (`inv6` = 0), the divisions decide.
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t quantise8(const float2 (&x)[4], float m, float scale, float inv6,
                                              uint32_t& sf) {
  constexpr float kUp = 1.f + 0x1p-20f, kDown = 1.f - 0x1p-20f;
  const float t = m * inv6;
  sf = f32_to_e4m3(t * kUp);
  if (inv6 == 0.f || sf != f32_to_e4m3(t * kDown)) sf = f32_to_e4m3(__fdiv_rn(__fdiv_rn(m, 6.0f), scale));
  const float den = __fmul_rn(e4m3_to_f32(sf), scale);
  if (den == 0.f) return 0u;
  const float inv = rcp_approx(den);
  uint32_t up = 0, down = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 y = mul2(x[i], make_float2(inv, inv));
    const float2 hi = mul2(y, make_float2(kUp, kUp)), lo = mul2(y, make_float2(kDown, kDown));
    up |= f32x2_to_e2m1x2(hi.x, hi.y) << (8 * i);
    down |= f32x2_to_e2m1x2(lo.x, lo.y) << (8 * i);
  }
  if (inv6 == 0.f || up != down) {
    up = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      up |= f32x2_to_e2m1x2(__fdiv_rn(x[i].x, den), __fdiv_rn(x[i].y, den)) << (8 * i);
  }
  // codes whose magnitude is zero are +0
  const uint32_t mag = (up | (up >> 1) | (up >> 2)) & 0x11111111u;
  return up & (0x77777777u | (mag << 3));
}

template <int D, bool kAppend, bool kInter, int STEPS>
__global__ void __launch_bounds__(kWarps * 32, STEPS == 1 ? 8 : kAppend ? 5 : 6)
prologue_kernel(const __grid_constant__ KernelArgs p) {
  constexpr int LPV = D / 8;        // lanes per head
  constexpr int VPW = 32 / LPV;     // heads that a warp holds
  const Geom& g = p.g;
  const PrologueArgs& a = p.a;
  const int lane = threadIdx.x & 31;
  const int l = lane % LPV, e0 = 8 * l;   // the lane's first element
  const uint32_t T = (uint32_t)g.B * (uint32_t)g.R;
  pdl_wait();
  pdl_trigger();

  // A turn: row, queries (or keys and values) and the lane's first head.
  struct Turn {
    uint32_t row;
    bool query;
    int head;
  };
  auto turn_of = [&](uint32_t row, uint32_t i) {     // (the row's turn i)
    Turn t;
    t.row = row;
    t.query = i < (uint32_t)p.turns_q;
    t.head = (int)(i - (t.query ? 0u : (uint32_t)p.turns_q)) * (VPW * STEPS) + lane / LPV;
    return t;
  };
  const int kvs = kAppend ? 2 * g.Hkv : g.Hkv;      // keys and values of a row
  const int psh = 31 - __clz(g.P);                  // log2 of the page size
  uint4 coming[STEPS];
  auto request = [&](const Turn& t) {
    const int heads = t.row >= T ? 0 : t.query ? g.Hq : kvs;
    if (!kAppend || t.query) {
      const __nv_bfloat16* src = t.query ? a.q + t.row * a.q_stride : a.k + t.row * a.k_stride;
      src += t.head * D + e0;
#pragma unroll
      for (int i = 0; i < STEPS; ++i)
        coming[i] = t.head + i * VPW < heads ? *reinterpret_cast<const uint4*>(src + i * VPW * D)
                                             : make_uint4(0u, 0u, 0u, 0u);
    } else {
      const __nv_bfloat16* k = a.k + t.row * a.k_stride + e0;
      const __nv_bfloat16* v = a.v + t.row * a.v_stride + e0;
#pragma unroll
      for (int i = 0; i < STEPS; ++i) {
        const int hd = t.head + i * VPW;
        const __nv_bfloat16* src = hd < g.Hkv ? k + hd * D : v + (hd - g.Hkv) * D;
        coming[i] = hd < heads ? *reinterpret_cast<const uint4*>(src) : make_uint4(0u, 0u, 0u, 0u);
      }
    }
  };

  float2 w[4];          // the lane's weights, of the queries or of the keys
  int w_of = -1;
  // turns of all rows one behind the other, this warp's `step` apart (2^24 rows of at most 2^8)
  const uint32_t turns = p.turns, item = blockIdx.x * kWarps + (threadIdx.x >> 5), step = gridDim.x * kWarps;
  uint32_t row = item / turns, at = item - row * turns;
  const uint32_t step_rows = STEPS > 1 ? step / turns : 0u, step_at = STEPS > 1 ? step - step_rows * turns : 0u;
  Turn now = turn_of(row, at);
  request(now);
  while (now.row < T) {
    const uint32_t r = now.row;
    const bool query = now.query;
    const int head0 = now.head, heads = query ? g.Hq : kvs;
    const int first = head0 - lane / LPV, left = heads - first;   // of the warp: steps past it hold nothing
    const int turning = query || !kAppend ? left : g.Hkv - first;   // and steps past this only values
    uint4 raws[STEPS];
#pragma unroll
    for (int i = 0; i < STEPS; ++i) raws[i] = coming[i];
    if (STEPS > 1) {
      row += step_rows;
      at += step_at;
      if (at >= turns) {
        at -= turns;
        ++row;
      }
      now = turn_of(row, at);
      request(now);
    } else {
      now.row = T;
    }

    // the row's slot in the cache
    size_t page_row = 0;
    int slot = 0;
    bool has_slot = false;
    if (kAppend && !query) {
      const uint32_t b = r / (uint32_t)g.R;
      const long long pos = (long long)a.seqlens[b] - g.R + (int)(r - b * (uint32_t)g.R);
      if (pos >= 0 && pos < (long long)g.MB * g.P) {
        const int page = a.page_table[(size_t)b * g.MB + ((int)pos >> psh)];
        slot = (int)pos & (g.P - 1);
        has_slot = page >= 0 && page < g.NP;
        page_row = (size_t)(has_slot ? page : 0);
      }
      // the index key, with the row's first keys: 16 lanes x 4 B
      if (head0 < VPW && has_slot && lane < kIndexDim / 4) {
        const uint32_t x = *reinterpret_cast<const uint32_t*>(a.ik + (size_t)r * kIndexDim + 4 * lane);
        *reinterpret_cast<uint32_t*>(a.ik_pool + ((page_row << psh) + slot) * kIndexDim + 4 * lane) = x;
      }
    }

    {
      // the lane's cos and sin: o = y c + partner s, with the sign of the first
      // half's sine in s
      const int rot = p.nr.rot, h = rot >> 1;
      const bool turned = e0 < rot;
      int partner = lane;
      float2 c[4], s[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) c[i] = s[i] = make_float2(0.f, 0.f);
      if (turned) {
        const float2* row = reinterpret_cast<const float2*>(a.cs) + (size_t)r * h;
        if (kInter) {
          const float4* row4 = reinterpret_cast<const float4*>(row + (e0 >> 1));
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float4 t = __ldg(row4 + i);
            c[2 * i] = make_float2(t.x, t.x);
            s[2 * i] = make_float2(-t.y, t.y);
            c[2 * i + 1] = make_float2(t.z, t.z);
            s[2 * i + 1] = make_float2(-t.w, t.w);
          }
        } else {
          const bool first = e0 < h;
          partner = first ? lane + h / 8 : lane - h / 8;
          const float4* row4 = reinterpret_cast<const float4*>(row + (first ? e0 : e0 - h));
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 t = __ldg(row4 + i);
            c[i] = make_float2(t.x, t.z);
            s[i] = first ? make_float2(-t.y, -t.w) : make_float2(t.y, t.w);
          }
        }
      }
      const __nv_bfloat16* weight = query ? a.q_weight : a.k_weight;
      if (weight && (int)query != w_of) {
        w_of = query;
        unpack8(__ldg(reinterpret_cast<const uint4*>(weight + e0)), w);
        if (p.nr.plus_one) {
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = add2(make_float2(1.f, 1.f), w[i]);
        }
      }

      // Sums of squares, neighbours first: eight in the lane, then lanes 1, 2, 4, ...
      // apart.  Four steps' sums are folded into one another on the way (a lane passes on
      // the sums it does not keep), so that lane i ends with that of step i mod 4, and one
      // square root and division serve all four.
      float rms[STEPS];
      if (weight) {
        float ss[STEPS];
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
          ss[i] = 0.f;
          if ((STEPS > 1 || kAppend) && i * VPW >= turning) continue;
          float2 x[4];
          unpack8(raws[i], x);
#pragma unroll
          for (int k = 0; k < 4; ++k) x[k] = mul2(x[k], x[k]);
          const float2 u = add2(make_float2(x[0].x, x[1].x), make_float2(x[0].y, x[1].y));
          const float2 v = add2(make_float2(x[2].x, x[3].x), make_float2(x[2].y, x[3].y));
          const float2 t = add2(make_float2(u.x, v.x), make_float2(u.y, v.y));
          ss[i] = __fadd_rn(t.x, t.y);
        }
        float sum = ss[0];
        if constexpr (STEPS == 4) {
          const bool odd = lane & 1, upper = lane & 2;
          const float k01 = odd ? ss[1] : ss[0], g01 = odd ? ss[0] : ss[1];
          const float k23 = odd ? ss[3] : ss[2], g23 = odd ? ss[2] : ss[3];
          const float s01 = __fadd_rn(k01, __shfl_xor_sync(0xffffffffu, g01, 1));
          const float s23 = __fadd_rn(k23, __shfl_xor_sync(0xffffffffu, g23, 1));
          sum = __fadd_rn(upper ? s23 : s01, __shfl_xor_sync(0xffffffffu, upper ? s01 : s23, 2));
        }
#pragma unroll
        for (int k = STEPS == 4 ? 4 : 1; k < LPV; k <<= 1)
          sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, k));
        const float inv = __fdiv_rn(1.f, __fsqrt_rn(__fadd_rn(sum * (1.f / D), p.nr.eps)));
#pragma unroll
        for (int i = 0; i < STEPS; ++i)
          rms[i] = STEPS == 4 ? __shfl_sync(0xffffffffu, inv, (lane & ~(LPV - 1)) + i) : inv;
      }

      __nv_bfloat16* out = query ? a.q_out : a.k_out;
      if (!kAppend || query) out += ((size_t)r * heads + head0) * D + e0;
#pragma unroll
      for (int i = 0; i < STEPS; ++i) {
        if ((STEPS > 1 || kAppend) && i * VPW >= turning) break;
        float2 y[4];
        unpack8(raws[i], y);
        if (weight) {
          const float2 m = make_float2(rms[i], rms[i]);
#pragma unroll
          for (int k = 0; k < 4; ++k) y[k] = mul2(mul2(y[k], m), w[k]);
        }
        if (kInter) {
          if (turned) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              y[k] = turn2(y[k], c[k], make_float2(y[k].y, y[k].x), s[k]);
          }
        } else if (rot) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 t = make_float2(__shfl_sync(0xffffffffu, y[k].x, partner),
                                         __shfl_sync(0xffffffffu, y[k].y, partner));
            if (turned) y[k] = turn2(y[k], c[k], t, s[k]);
          }
        }
        if (!kAppend || query || head0 + i * VPW < g.Hkv) raws[i] = pack8(y);   // (values stay)
        if ((!kAppend || query) && head0 + i * VPW < heads)
          *reinterpret_cast<uint4*>(out + i * VPW * D) = raws[i];
      }
    }
    if constexpr (kAppend) {
      if (query) continue;

      // keys and values: blocks of 16 (two lanes) to e2m1 codes and an e4m3 scale,
      // as the token store quantises them
#pragma unroll
      for (int i = 0; i < STEPS; ++i) {
        if (STEPS > 1 && i * VPW >= left) break;
        float2 x[4];
        unpack8(raws[i], x);
        float m = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) m = fmaxf(m, fmaxf(fabsf(x[k].x), fabsf(x[k].y)));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        if (head0 + i * VPW < heads && has_slot) {
          const bool val = head0 + i * VPW >= g.Hkv;
          uint8_t* pool = val ? a.v_pool : a.k_pool;
          uint8_t* sfp = val ? a.v_sf : a.k_sf;
          uint32_t sf;
          const uint32_t codes = quantise8(x, m, val ? a.v_scale : a.k_scale, val ? p.v_inv6 : p.k_inv6, sf);
          const size_t row = (((page_row * g.Hkv + (head0 + i * VPW - (val ? g.Hkv : 0))) << psh)) + slot;
          if (QSA_IN_BOUNDS(row < (size_t)g.NP * g.Hkv * g.P, kChkRow)) {
            *reinterpret_cast<uint32_t*>(pool + row * (D / 2) + 4 * l) = codes;
            if (!(l & 1)) sfp[row * (D / 16) + (l >> 1)] = (uint8_t)sf;
          }
        }
        __syncwarp();
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Cache rows read back: eight elements (4 code bytes, one scale) of a key and of its
// value per lane, for ROWS rows at once: three loads depend on one another (length, page,
// codes), so what is in flight decides: waiting for loads is
// its largest stall, 3.2 cycles an instruction (16 code bytes a lane would be fewer and wider
// loads).  A CTA has neighbouring rows of one head, which
// are neighbours in their page.
// ---------------------------------------------------------------------------
template <int D, int ROWS>
__global__ void __launch_bounds__(kWarps * 32)
load_tokens_kernel(Geom g, const int32_t* __restrict__ page_table,
                   const int32_t* __restrict__ seqlens, const uint8_t* __restrict__ k_pool,
                   const uint8_t* __restrict__ k_sf, const uint8_t* __restrict__ v_pool,
                   const uint8_t* __restrict__ v_sf, float k_scale, float v_scale,
                   __nv_bfloat16* __restrict__ k_out, __nv_bfloat16* __restrict__ v_out) {
  const int l = threadIdx.x, psh = 31 - __clz(g.P), head = blockIdx.y;
  const uint32_t r0 = blockIdx.x * (blockDim.y * ROWS) + threadIdx.y, rows = (uint32_t)g.B * (uint32_t)g.R;
  pdl_wait();
  pdl_trigger();
  int page[ROWS], slot[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const uint32_t r = r0 + i * blockDim.y, b = r / (uint32_t)g.R;
    page[i] = -1;
    if (r >= rows) continue;
    const long long pos = (long long)seqlens[b] - g.R + (int)(r - b * (uint32_t)g.R);
    slot[i] = (int)pos & (g.P - 1);
    if (pos >= 0 && pos < (long long)g.MB * g.P)
      page[i] = page_table[(size_t)b * g.MB + ((int)pos >> psh)];
    if (page[i] >= g.NP) page[i] = -1;
  }
  uint32_t codes[ROWS][2], sfs[ROWS][2];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const size_t row = page[i] < 0 ? 0 : (((size_t)page[i] * g.Hkv + head) << psh) + slot[i];
    if (!QSA_IN_BOUNDS(row < (size_t)g.NP * g.Hkv * g.P, kChkLoad)) page[i] = -1;
    if (page[i] < 0) continue;
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      codes[i][v] = *reinterpret_cast<const uint32_t*>((v ? v_pool : k_pool) + row * (D / 2) + 4 * l);
      sfs[i][v] = (v ? v_sf : k_sf)[row * (D / 16) + (l >> 1)];
    }
  }
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    if (page[i] < 0) continue;
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      const float sf = e4m3_to_f32(sfs[i][v]), scale = v ? v_scale : k_scale;
      float2 x[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uint32_t h2 = e2m1x2_to_f16x2((codes[i][v] >> (8 * u)) & 0xFFu);
        // code * block scale is exact in fp32; the tensor scale rounds once
        const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&h2));
        x[u] = make_float2(__fmul_rn(y.x * sf, scale), __fmul_rn(y.y * sf, scale));
      }
      __nv_bfloat16* out = v ? v_out : k_out;
      *reinterpret_cast<uint4*>(out + ((size_t)(r0 + i * blockDim.y) * g.Hkv + head) * D + 8 * l) = pack8(x);
    }
  }
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
  const long long most = 16 * sm_count();   // (what is resident takes turns)
  return launch(rope_rows_kernel, dim3((unsigned)(ctas < most ? ctas : most)), block, pdl, stream,
                g.R, T, rope, seqlens, positions, reinterpret_cast<float2*>(cs));
}

cudaError_t launch_prologue(const Geom& g, const NormRope& nr, const PrologueArgs& a, bool pdl,
                            cudaStream_t stream) {
  const bool append = a.v != nullptr;
  KernelArgs p;
  p.g = g;
  p.nr = nr;
  p.a = a;
  auto inverse = [](float scale) {
    const float inv = 1.f / (6.f * scale);
    return inv > 0x1p-100f && inv < 0x1p100f ? inv : 0.f;
  };
  p.k_inv6 = append ? inverse(a.k_scale) : 0.f;
  p.v_inv6 = append ? inverse(a.v_scale) : 0.f;
  const int vpw = g.D == 128 ? 2 : 1;
  const long long T = (long long)g.B * g.R;
  const int total = (a.q ? g.Hq : 0) + (append ? 2 : 1) * g.Hkv;   // heads per row
  // Few rows: a turn of one step, for the shortest chain; many rows: four steps
  // share the row's cos and sin and one square root (40 heads of 128: 64 rows 2.1 and 2.9 us
  // with one and four, 256 rows, 5120 single turns, 3.4 both, 512 rows 5.4 and 5.0, 2048 rows
  // 16.9 and 11.2).
  const int sms = sm_count(), steps = T * total / vpw > sms * 40 ? 4 : 1, per = vpw * steps;
  p.turns_q = a.q ? (g.Hq + per - 1) / per : 0;
  p.turns = p.turns_q + ((append ? 2 : 1) * g.Hkv + per - 1) / per;
  const long long items = T * p.turns;
  auto launch_it = [&]<int D, bool kAppend, bool kInter>() {
    auto* kern = steps == 4 ? prologue_kernel<D, kAppend, kInter, 4> : prologue_kernel<D, kAppend, kInter, 1>;
    // many rows: six CTAs per SM stay and take turns, or five of the append, which needs more
    // registers (two context chunks, norms: 40.4 us with six, 42.4 with five; append 58.1, 56.8)
    const long long ctas = (items + kWarps - 1) / kWarps, most = (kAppend ? 5 : 6) * sms;
    return launch(kern, dim3((unsigned)(steps == 4 && ctas > most ? most : ctas)), dim3(kWarps * 32),
                  pdl, stream, p);
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
  const dim3 block(g.D / 8, kWarps * 32 / (g.D / 8));
  const unsigned rows = (unsigned)g.B * (unsigned)g.R;
  // Few rows: one per thread, for the shortest chain (192 rows of 4 heads: 4.1 us, 5.8 with
  // four); many: four, for more in flight (8188 rows of 2 heads at head_dim 256: 7.3 us, 10.7
  // with one).
  const bool many = (long long)rows * g.Hkv > sm_count() * 16 * (long long)block.y;
  const unsigned per = block.y * (many ? 4 : 1);
  auto* kern = many ? (g.D == 256 ? load_tokens_kernel<256, 4> : load_tokens_kernel<128, 4>)
                    : (g.D == 256 ? load_tokens_kernel<256, 1> : load_tokens_kernel<128, 1>);
  return launch(kern, dim3((rows + per - 1) / per, g.Hkv), block, pdl, stream, g,
                page_table, seqlens, k_pool, k_sf, v_pool, v_sf, k_scale, v_scale,
                reinterpret_cast<__nv_bfloat16*>(k_out), reinterpret_cast<__nv_bfloat16*>(v_out));
}

}  // namespace qsa

QSA_BOUNDS_READER(bounds_word_prologue)
