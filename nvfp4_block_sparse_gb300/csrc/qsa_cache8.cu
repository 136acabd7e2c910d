// qsa_cache8.cu -- the 8-bit cache's rows: appended with a scale for each block
// of 16 tokens and KV head, and read back.
//
//   e    = least integer in [-32, 64] with max |x| <= 448 2^e over the block's new
//          tokens, not less than the block's former one where tokens of it stay
//   code = e4m3(x 2^-e)
//
// Powers of two, because a block fills token by token: when a later token raises
// the scale, the codes that are there are rounded again, and dividing a floating-point
// code by a power of two is exact until it becomes subnormal.  e4m3 has the same
// relative steps in all its binades, so a scale between powers of two would buy
// nothing but the last binade's unused quarter.  The range of e: the attention over the
// cache weighs V's codes by exp(z) 2^e in fp32, and with exponents at most 96 apart no
// weight that counts is lost.
//
// Work: a CTA has up to 16 neighbouring rows.  A row that is the first of its request's
// new rows in its block leads the block, and a warp takes the block's new rows (up to 16, wherever they
// lie) of one head's keys or values: all requested at once, so that their largest magnitude is
// there before the first is rounded, without reading anything twice.  So a block is
// written by one warp whatever the rows' number, nothing waits for anybody else, and
// requests of any lengths, packed or not, are the same to it.
// Bound by the rows' bytes: 2 in and 1 out per element, for few rows by two chains of length, page and
// row.  Measured (GB300, both calls behind one another on the GPU): 6 packed prompts of 700 to 2047
// tokens, 2 heads of 256, append and read-back 15.7 us for 52.9 MB, of which the append takes the larger
// half (a block's 16 rows are 127 registers of a thread: a quarter of the SM's warps; 0.8 of its time
// it waits for the one look at lengths and pages and the one at the rows); 48 requests of 4 rows 5.2 us.
#include "qsa_common.cuh"

namespace qsa {
namespace {

// Bounds-check codes (reported by bounds-checked builds only).
[[maybe_unused]] constexpr int kChkRow = 0xB01;    // append: pool row out of range
[[maybe_unused]] constexpr int kChkLoad = 0xB02;   // read-back: pool row out of range

constexpr int kBlock = 16;            // tokens per scale
constexpr int kRows = 16;             // rows of a CTA, at most
constexpr int kLeastExp = 127 - 32, kMostExp = 127 + 64;

// Where row r of the call lies.
struct Place {
  int page, slot;      // page < 0: it has no slot
  int nth, count;      // its number among the request's rows; how many those are
};

__device__ __forceinline__ Place place_of(const Geom& g, const Cache8Args& a, uint32_t r) {
  Place p;
  p.page = -1;
  p.slot = p.nth = p.count = 0;
  int b;
  if (a.cu) {
    // the last request whose rows begin at or before r
    int lo = 0, hi = g.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(a.cu + mid) <= (int)r) lo = mid;
      else hi = mid;
    }
    b = lo;
    const int first = __ldg(a.cu + b), end = __ldg(a.cu + b + 1);
    if (first < 0 || first > (int)r || end <= (int)r || end > a.rows) return p;
    p.nth = (int)r - first;
    p.count = end - first;
  } else {
    b = (int)(r / (uint32_t)g.R);
    p.nth = (int)(r - (uint32_t)b * (uint32_t)g.R);
    p.count = g.R;
  }
  const long long pos = (long long)a.seqlens[b] - p.count + p.nth;
  const int psh = 31 - __clz(g.P);
  if (pos < 0 || pos >= (long long)g.MB * g.P) return p;
  const int page = a.page_table[(size_t)b * g.MB + ((int)pos >> psh)];
  p.slot = (int)pos & (g.P - 1);
  if (page >= 0 && page < g.NP) p.page = page;
  return p;
}

__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(lo), "f"(hi));
  return r;
}

// 2^(e - 127) for 1 <= e <= 254.
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)e << 23); }

template <int D>
__global__ void __launch_bounds__(256)
store8_kernel(const __grid_constant__ Geom g, const __grid_constant__ Cache8Args a, int rows) {
  constexpr int LPT = D / 8;             // lanes per token, eight elements each
  constexpr int TPS = 32 / LPT;          // tokens per step of a warp
  constexpr int STEPS = kBlock / TPS;
  __shared__ int4 s_lead[kRows];         // page, slot, rows, first row
  __shared__ int s_leads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_trigger();
  if (warp == 0) {
    const uint32_t r = blockIdx.x * (uint32_t)rows + lane;
    Place p;
    p.page = -1;
    if (lane < rows && r < (uint32_t)a.rows) p = place_of(g, a, r);
    const bool leads = p.page >= 0 && (p.nth == 0 || (p.slot & (kBlock - 1)) == 0);
    const uint32_t which = __ballot_sync(0xffffffffu, leads);
    if (leads)
      s_lead[__popc(which & ((1u << lane) - 1u))] =
          make_int4(p.page, p.slot, min(kBlock - (p.slot & (kBlock - 1)), p.count - p.nth), (int)r);
    if (lane == 0) s_leads = __popc(which);
  }
  __syncthreads();
  const int psh = 31 - __clz(g.P), l = lane % LPT, sub = lane / LPT;
  const int items = s_leads * 2 * g.Hkv;
  for (int item = warp; item < items; item += 8) {
    const int which = item / (2 * g.Hkv), rest = item - which * 2 * g.Hkv;
    const bool val = rest >= g.Hkv;
    const int head = val ? rest - g.Hkv : rest;
    const int4 at = s_lead[which];
    const int slot = at.y, count = at.z;
    const __nv_bfloat16* src = (val ? a.v : a.k) + (size_t)at.w * (val ? a.v_stride : a.k_stride) +
                               (size_t)head * D + 8 * l;
    const size_t stride = (size_t)(val ? a.v_stride : a.k_stride);
    uint4 raw[STEPS];
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const int t = i * TPS + sub;
      raw[i] = t < count ? *reinterpret_cast<const uint4*>(src + t * stride) : make_uint4(0u, 0u, 0u, 0u);
    }
    const size_t row0 = ((((size_t)at.x * g.Hkv + head) << psh)) + (slot & ~(kBlock - 1));
    if (!QSA_IN_BOUNDS(row0 + kBlock <= (size_t)g.NP * g.Hkv * g.P, kChkRow)) continue;
    uint8_t* exp_at = (val ? a.v_exp : a.k_exp) + row0 / kBlock;
    uint8_t* pool = (val ? a.v_pool : a.k_pool) + row0 * D + 8 * l;
    const int off = slot & (kBlock - 1);     // tokens that stay
    const int before = off ? min(max((int)*exp_at, kLeastExp), kMostExp) : kLeastExp;

    // the largest finite magnitude, as bf16 bits (ordered as integers are)
    uint32_t top = 0u;
    auto words = [&](const uint4& r, int w) { return w == 0 ? r.x : w == 1 ? r.y : w == 2 ? r.z : r.w; };
#pragma unroll
    for (int i = 0; i < STEPS; ++i)
#pragma unroll
      for (int w = 0; w < 4; ++w) top = __vmaxu2(top, words(raw[i], w) & 0x7FFF7FFFu);
    uint32_t m = max(top & 0xFFFFu, top >> 16);
    m = __reduce_max_sync(0xffffffffu, m);
    const bool odd = m >= 0x7F80u;     // something is not finite: it becomes NaN, the others decide
    if (odd) {
      m = 0u;
#pragma unroll
      for (int i = 0; i < STEPS; ++i)
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint32_t x = words(raw[i], w) & 0x7FFF7FFFu;
          if ((x & 0xFFFFu) < 0x7F80u) m = max(m, x & 0xFFFFu);
          if ((x >> 16) < 0x7F80u) m = max(m, x >> 16);
        }
      m = __reduce_max_sync(0xffffffffu, m);
    }
    // 448 = 1.75 2^8
    const int least = (int)(m >> 7) - 8 + ((m & 0x7Fu) > 0x60u ? 1 : 0);
    const int e = min(max(max(least, kLeastExp), before), kMostExp);
    const float down = pow2(254 - e);        // 2^(127 - e)

    if (e > before && off) {
      const float by = pow2(127 + before - e);
#pragma unroll 4
      for (int t = sub; t < off; t += TPS) {
        uint2* p = reinterpret_cast<uint2*>(pool + (size_t)t * D);
        const uint2 c = *p;
        uint32_t o[2];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const uint32_t x = w ? c.y : c.x, a2 = e4m3x2_to_f16x2(x & 0xFFFFu), b2 = e4m3x2_to_f16x2(x >> 16);
          const float2 u = __half22float2(*reinterpret_cast<const __half2*>(&a2));
          const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&b2));
          o[w] = f32x2_to_e4m3x2(u.x * by, u.y * by) | f32x2_to_e4m3x2(v.x * by, v.y * by) << 16;
        }
        *p = make_uint2(o[0], o[1]);
      }
    }
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const int t = i * TPS + sub;
      if (t >= count) continue;
      uint32_t o[2] = {0u, 0u};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint32_t x = words(raw[i], w);
        float lo = __uint_as_float(x << 16), hi = __uint_as_float(x & 0xFFFF0000u);
        if (odd) {
          const float nan = __uint_as_float(0x7FC00000u);
          if ((x & 0x7F80u) == 0x7F80u) lo = nan;
          if ((x & 0x7F800000u) == 0x7F800000u) hi = nan;
        }
        o[w >> 1] |= f32x2_to_e4m3x2(lo * down, hi * down) << (16 * (w & 1));
      }
      *reinterpret_cast<uint2*>(pool + (size_t)(off + t) * D) = make_uint2(o[0], o[1]);
    }
    if (lane == 0) *exp_at = (uint8_t)e;
    __syncwarp();
  }
}

// Read-back: items (row, head, key or value) of up to 16 rows, D / 8 lanes each, UNROLL of them
// on their way at a time.
template <int D, int UNROLL>
__global__ void __launch_bounds__(256)
load8_kernel(const __grid_constant__ Geom g, const __grid_constant__ Cache8Args a, int rows) {
  constexpr int LPT = D / 8, kAtOnce = 256 / LPT;
  __shared__ int2 s_place[kRows];
  pdl_wait();
  pdl_trigger();
  if (threadIdx.x < rows) {
    const uint32_t r = blockIdx.x * (uint32_t)rows + threadIdx.x;
    Place p;
    p.page = -1;
    p.slot = 0;
    if (r < (uint32_t)a.rows) p = place_of(g, a, r);
    s_place[threadIdx.x] = make_int2(p.page, p.slot);
  }
  __syncthreads();
  const int psh = 31 - __clz(g.P), l = threadIdx.x % LPT;
  const int per = 2 * g.Hkv, items = rows * per;
  for (int i0 = threadIdx.x / LPT; i0 < items; i0 += UNROLL * kAtOnce) {
    uint2 codes[UNROLL];
    int exps[UNROLL];
    __nv_bfloat16* to[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int item = i0 + u * kAtOnce;
      to[u] = nullptr;
      if (item >= items) continue;
      const int row = item / per, rest = item - row * per;
      const bool val = rest >= g.Hkv;
      const int head = val ? rest - g.Hkv : rest;
      const int2 at = s_place[row];
      if (at.x < 0) continue;
      const size_t src = (((size_t)at.x * g.Hkv + head) << psh) + at.y;
      if (!QSA_IN_BOUNDS(src < (size_t)g.NP * g.Hkv * g.P, kChkLoad)) continue;
      codes[u] = *reinterpret_cast<const uint2*>((val ? a.v_pool : a.k_pool) + src * D + 8 * l);
      exps[u] = (val ? a.v_exp : a.k_exp)[src / kBlock];
      to[u] = (val ? a.v_out : a.k_out) +
              ((size_t)(blockIdx.x * (uint32_t)rows + row) * g.Hkv + head) * D + 8 * l;
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      if (!to[u]) continue;
      const float s = pow2(min(max(exps[u], kLeastExp), kMostExp));   // (as attention takes them)
      uint32_t o[4];
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t x = (w & 2 ? codes[u].y : codes[u].x) >> (16 * (w & 1));
        const uint32_t h2 = e4m3x2_to_f16x2(x & 0xFFFFu);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
        const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * s, f.y * s);
        o[w] = *reinterpret_cast<const uint32_t*>(&b);
      }
      *reinterpret_cast<uint4*>(to[u]) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

}  // namespace

cudaError_t launch_cache8(const Geom& g, const Cache8Args& a, bool append, bool pdl,
                          cudaStream_t stream) {
  // Rows per CTA: as many as leave every SM eight CTAs, so that a decode step's few rows are
  // spread (48 requests of 4 rows: 5.2 us; in CTAs of 16 rows 12 SMs would do them) and a prompt's
  // blocks are found by one look per block.
  const long long sms = sm_count();
  int rows = 1;
  while (rows < kRows && a.rows > rows * sms * 8) rows *= 2;
  auto* kern = append ? (g.D == 256 ? store8_kernel<256> : store8_kernel<128>)
                      : (g.D == 256 ? load8_kernel<256, 4> : load8_kernel<128, 4>);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.rows + rows - 1) / rows));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, g, a, rows);
}

}  // namespace qsa

QSA_BOUNDS_READER(bounds_word_cache8)
