// qsa_dense.cuh -- what the two dense attention kernels share: the units of
// work, their even division over the CTAs, and the records of a unit that is
// divided between CTAs.
//
// A unit is (request b, tile t of its query vectors, KV head).  The R*G query
// vectors of a request and KV head are numbered row j, head h -> j*G + h; tile
// t holds vectors [t*VT, (t+1)*VT).  A unit walks the chunks of TOK tokens from
// the first token that its first row sees to the last that its last row sees;
// one with no token has one chunk all the same, so that somebody writes its
// zeros.  The units' chunks, one behind the other, are divided evenly over the
// CTAs of the grid by the requests' actual lengths: CTA i takes chunks
// [i*share, (i+1)*share).  So every CTA ends at about the same time whatever
// the lengths, and a single long request still uses the whole GPU.  Starting a unit
// costs as much as some chunks do, so each counts with `lead` chunks more, ahead of its
// own, that hold nothing.
//
// A unit inside one CTA is written out by it.  A unit that crosses CTAs leaves
// a record (base, sum, unscaled output per vector) from each of them: in slot 1
// of the CTA where it begins, in slot 0 of the others.  The CTA where a unit
// ends writes its descriptor, and a second kernel joins the records in the
// CTAs' order, whatever order they ended in.  Descriptors go by unit, or, where
// there are more units than CTAs, by the CTA where the divided unit ends (there
// is at most one).  The decode kernel's records are small, and the CTA that is
// last to finish with a unit joins them itself, in the same order (a ticket per
// CTA where a divided unit ends, which every call leaves at zero).
#pragma once

#include "qsa_common.cuh"

namespace qsa {
namespace dense {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// (A vector that sees nothing has a sum of exactly 0, and lse = -inf; a NaN in its queries or
// keys makes its sum NaN, which out and lse pass on.)
// The softmax base before a vector has seen a token: low enough for every
// logit to move it, finite so that differences with -inf stay -inf.
constexpr float kNoBase = -1e30f;
// Weights are fp16, of 11 bits from 2^-14 to 65504.  A vector's base (log2) moves when a logit
// exceeds it by more than kHeadroom, near the upper end, and then to kBelow below that logit:
// so weights down to 2^-22 of the largest keep all their bits (15 nats: a first token that takes
// nearly everything leaves the others theirs), smaller ones lose them and those below 2^-33
// count as zero against V.  The bits between the two are what later logits may rise by without
// another move, which in the tile kernel waits for O and rewrites it: windowed verify 44.5, 44.5,
// 48, 58 us and the context 648, 643, 658, 722 with 0, 7, 10, 14 below and a headroom of 15.
constexpr float kHeadroom = 15.9f;
constexpr float kBelow = 8.f;

// Two weights as fp16.  Their exponents' arguments are a logit's exact product less a rounded
// base, off by the base's fp32 step: with logits of 2^20 and more a weight just inside the
// headroom would pass 65504, and stays there instead.
__device__ __forceinline__ uint32_t pack_weights(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Which of four e4m3 codes are NaN: the upper bits of their bytes.  And the codes with those as zeros.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }
__device__ __forceinline__ uint32_t without_nan(uint32_t w) { return w & ~((nan_codes(w) >> 7) * 0xFFu); }

struct Shape {
  Geom g;
  int G;         // query heads per KV head
  uint32_t g_mul;   // ceil(2^32 / G) for G > 1: divides vector numbers (row_of)
  int vt;        // query vectors per tile
  int tiles;     // tiles per request
  int tok_sh;    // log2 of the tokens per chunk
  int window;    // tokens a row looks back over; 0: all
  int least;     // chunks a CTA takes at least
  int lead;      // chunks that a unit counts beyond its own
  int ctas;      // CTAs of the grid
  int by_unit;   // descriptors go by unit (else by CTA)
};

// A divided unit's descriptor.
struct Desc {
  int b, tile, kvh;   // b < 0: nothing to join
  int first, last;    // CTAs where the unit begins and ends
  int pad[3];
};

struct Work {
  const __nv_bfloat16* q;
  const uint8_t *k_pool, *k_sf, *v_pool, *v_sf;   // (8-bit pages: k_sf and v_sf are the exponents)
  float v_scale;
  float z_mant;      // k_scale sm_scale log2(e) = z_mant 2^z_exp, z_mant in [1/2, 1)
  int z_exp;
  const int32_t *page_table, *seqlens;
  const float* sinks;
  __nv_bfloat16* out;
  float* lse;
  int* status;
  Desc* desc;        // [units or CTAs]
  int* tickets;      // [CTAs]
  float* records;    // [CTAs][2][vt * (2 + D)]: bases, sums, outputs ([vt][D], or of the tile
                     // kernel [D/4][vt][4])
};

// Factor from the products of a vector scaled by 2^sq to its log2 logits.  The scales may be
// far apart in size, so their product and the power of two meet as exponents; kept a positive
// normal number, so that a logit masked by -inf stays -inf (logits that small are all alike).
__device__ __forceinline__ float logit_factor(const Work& w, int sq) {
  const int e = min(max(w.z_exp - sq, -252), 252), half = e >> 1;
  auto pow2 = [](int n) { return __uint_as_float((uint32_t)(n + 127) << 23); };
  return fminf(fmaxf(w.z_mant * pow2(half) * pow2(e - half), 0x1p-126f), 0x1.fffffep127f);
}

__host__ __device__ __forceinline__ size_t record_floats(int vt, int D) {
  return (size_t)vt * (2 + D);
}

// Row of query vector x, x / G: for x < R G <= 2^19 and G <= 128 the product with
// ceil(2^32 / G) is too large by less than x G < 2^32, so its upper half is exact.  (A division by
// a variable is some 40 dependent instructions, and a part's start had eight of them.)
__device__ __forceinline__ int row_of(const Shape& s, int x) {
  return s.G == 1 ? x : (int)__umulhi((uint32_t)x, s.g_mul);
}
// Request of a group (request, tile): nearly always there is one tile.
__device__ __forceinline__ int request_of(const Shape& s, int group) {
  return s.tiles == 1 ? group : (int)((uint32_t)group / (uint32_t)s.tiles);
}

__device__ __forceinline__ int first_seen(int n, int window) {
  return window > 0 && n > window ? n - window : 0;
}

// What the rows of a tile see of a request of length L.
struct Sight {
  int vec0, vecs;            // query vectors of the tile
  int n_all, n_least;        // tokens that the last / first row sees
  int lo_all, lo_most;       // first token that the first / last row sees
  int first, count;          // chunks; at least one (with no token: its zeros are written)
};

__device__ __forceinline__ Sight sight_of(const Shape& s, int L, int tile) {
  Sight v;
  const int cap = s.g.MB * s.g.P;
  v.vec0 = tile * s.vt;
  v.vecs = min(s.vt, s.g.R * s.G - v.vec0);
  v.n_all = visible_tokens(L, s.g.R, row_of(s, v.vec0 + v.vecs - 1), cap);
  v.n_least = visible_tokens(L, s.g.R, row_of(s, v.vec0), cap);
  v.lo_all = first_seen(v.n_least, s.window);
  v.lo_most = first_seen(v.n_all, s.window);
  v.first = 0;
  v.count = 1;
  if (v.n_all > v.lo_all) {
    v.first = v.lo_all >> s.tok_sh;
    v.count = ((v.n_all - 1) >> s.tok_sh) + 1 - v.first;
  }
  return v;
}

__device__ __forceinline__ int chunk_count(const Shape& s, const int32_t* seqlens, int group) {
  const int b = request_of(s, group);
  return sight_of(s, seqlens[b], group - b * s.tiles).count + s.lead;
}

// This CTA's part of the work, in the groups (request, tile) in order, each
// with Hkv units.  Called by all NTHR threads.
struct Span {
  long long begin, end;   // global chunks
  long long share;
  int group;              // group of `begin`
  long long group_at;     // global chunk where that group begins
};

template <int NTHR>
__device__ __forceinline__ Span plan_span(const Shape& s, const int32_t* seqlens, int cta,
                                          int ctas) {
  __shared__ long long s_warp[NTHR / 32];
  __shared__ long long s_at;
  __shared__ int s_group;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int groups = s.g.B * s.tiles;
  if (groups <= 32) {   // a lane per group, every warp for itself
    const uint32_t hkv = (uint32_t)s.g.Hkv;   // (counts to 2^17, heads to 2^8: within 32 bits)
    const uint32_t mine = lane < groups ? (uint32_t)chunk_count(s, seqlens, lane) * hkv : 0u;
    uint32_t x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    const uint32_t total = __shfl_sync(0xffffffffu, x, 31);
    const uint32_t share = max((total + (uint32_t)ctas - 1) / (uint32_t)ctas, (uint32_t)s.least);
    Span span;
    span.share = share;
    span.begin = (long long)share * cta;
    span.end = min((long long)total, span.begin + share);
    const uint32_t past = __ballot_sync(0xffffffffu, (long long)x > span.begin);
    span.group = past ? __ffs(past) - 1 : 0;
    span.group_at = __shfl_sync(0xffffffffu, x - mine, span.group);
    return span;
  }
  const int per = (groups + NTHR - 1) / NTHR;
  const int g0 = min(groups, tid * per), g1 = min(groups, g0 + per);
  long long mine = 0;
  for (int i = g0; i < g1; ++i) mine += chunk_count(s, seqlens, i);
  long long x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  long long before = x - mine, total = 0;
#pragma unroll
  for (int w = 0; w < NTHR / 32; ++w) {
    if (w < warp) before += s_warp[w];
    total += s_warp[w];
  }
  const int hkv = s.g.Hkv;
  total *= hkv;
  before *= hkv;
  Span span;
  span.share = (total + ctas - 1) / ctas;
  if (span.share < s.least) span.share = s.least;
  span.begin = span.share * cta;
  span.end = min(total, span.begin + span.share);
  if (span.begin < span.end && before <= span.begin && span.begin < before + mine * hkv) {
    long long at = before;
    int i = g0;
    for (; i < g1 - 1; ++i) {
      const long long c = (long long)chunk_count(s, seqlens, i) * hkv;
      if (span.begin < at + c) break;
      at += c;
    }
    s_at = at;
    s_group = i;
  }
  __syncthreads();
  span.group = s_group;
  span.group_at = s_at;
  return span;
}

// The part of one unit that a CTA does.
struct Seg : Sight {
  int b, tile, kvh;
  int L;
  int c_at, todo;            // chunks of the unit before this part, and in it
  bool begins, ends;         // the part holds the unit's first / last chunk
  int chunk0;                // first chunk of the part
};

// Walks a span's parts in order; every role of a CTA walks its own copy.
struct Cursor {
  long long at, end, group_at, unit_at;
  int group;
  __device__ __forceinline__ explicit Cursor(const Span& s)
      : at(s.begin), end(s.end), group_at(s.group_at), unit_at(0), group(s.group) {}
  __device__ __forceinline__ bool next(const Shape& s, const int32_t* seqlens, Seg& g) {
    while (at < end) {
      g.b = request_of(s, group);
      g.tile = group - g.b * s.tiles;
      g.L = seqlens[g.b];
      static_cast<Sight&>(g) = sight_of(s, g.L, g.tile);
      const uint32_t len = (uint32_t)(g.count + s.lead);
      const uint32_t in_group = (uint32_t)(at - group_at);   // (at most 2^18 chunks of 256 heads)
      g.kvh = (int)(in_group / len);
      const int from = (int)(in_group - (uint32_t)g.kvh * len);
      const int to = (int)min((long long)len, from + (end - at));
      unit_at = at - from;
      at += to - from;
      if (at == group_at + (long long)len * s.g.Hkv) {
        group_at = at;
        ++group;
      }
      g.c_at = max(from - s.lead, 0);
      g.todo = max(to - s.lead, 0) - g.c_at;
      g.begins = g.c_at == 0;
      g.ends = g.c_at + g.todo == g.count;
      g.chunk0 = g.first + g.c_at;
      if (g.todo > 0) return true;
    }
    return false;
  }
  // The CTAs where the unit of the last part begins and ends.
  __device__ __forceinline__ int first_cta(const Shape& s, long long share) const {
    return (int)((unit_at + s.lead) / share);
  }
  __device__ __forceinline__ int last_cta(const Shape& s, const Seg& g, long long share) const {
    return (int)((unit_at + s.lead + g.count - 1) / share);
  }
};

// By one thread, for every part that ends a unit (and, where descriptors go by
// CTA, first for the CTA: `none`).
__device__ __forceinline__ void describe(const Shape& s, const Work& w, const Span& span,
                                         const Cursor& cursor, const Seg& seg, int cta) {
  Desc d;
  d.b = seg.begins ? -1 : seg.b;
  d.tile = seg.tile;
  d.kvh = seg.kvh;
  d.first = cursor.first_cta(s, span.share);
  d.last = cta;
  if (s.by_unit)
    w.desc[(seg.b * s.tiles + seg.tile) * s.g.Hkv + seg.kvh] = d;
  else if (!seg.begins)
    w.desc[cta] = d;
}
__device__ __forceinline__ void describe_none(const Shape& s, const Work& w, int cta) {
  if (!s.by_unit) w.desc[cta].b = -1;
}

// The heads' part of a shape.
inline void set_heads(Shape* s, const Geom& g) {
  s->g = g;
  s->G = g.Hq / g.Hkv;
  s->g_mul = s->G == 1 ? 0u : (uint32_t)(((1ull << 32) + s->G - 1) / s->G);
}
// Units of a geometry, and how descriptors go.
inline long long unit_count(const Shape& s) { return (long long)s.g.B * s.tiles * s.g.Hkv; }
inline int desc_count(const Shape& s) { return s.by_unit ? (int)unit_count(s) : s.ctas; }

}  // namespace dense

// The tile kernel (qsa_dense_tile.cu): its units for this geometry, and its launch over NVFP4
// or (e8) 8-bit pages.
dense::Shape dense_tile_shape(const Geom& g, int window);
cudaError_t launch_dense_tile(const dense::Shape& s, const dense::Work& w, bool e8, cudaStream_t stream);
cudaError_t launch_dense_join(const dense::Shape& s, const dense::Work& w, cudaStream_t stream);
// The workspace's parts: status word, descriptors, records.
size_t dense_carve(const dense::Shape& s, void* workspace, dense::Work* w);

}  // namespace qsa
