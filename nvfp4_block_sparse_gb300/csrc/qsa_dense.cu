// qsa_dense.cu -- dense attention over the NVFP4 paged cache, few query
// vectors per KV head (decode and narrow verify rows), and the join of divided
// units.
//
// TensorRT-LLM PR #20937 ("GB300 perf work on
// qwen3_8_flash_next_nvfp4__sm_103__tp1"), What changes: NVFP4 GQA decode as
// split-K + merge; PR #20276 ("Qwen3.8-Flash-Next NVFP4 target"), Features
// table: uint8 e2m1 pages + e4m3 block scales.
//
//   z_t = sm_scale k_scale q.K_t,  out = v_scale sum_t exp(z_t) V_t / sum_t exp(z_t)
//
// The cache is read once (9/16 B per element), which bounds the work from
// below; per element there is one conversion and one product for half of it,
// so what the kernel does with its instructions decides how near it comes.
// Each warp works alone: it takes every W-th chunk of its CTA's part, streams
// it into its own shared-memory ring with asynchronous copies (no barrier with
// other warps, no wait on another thread), and keeps its own base, sum and
// output, which are joined at the end of the unit.
//
//   S^T = K Q^T    A = K: 16 tokens x 16 dims, e2m1 -> fp16 in registers times
//                  the block scale (exact), B = Q: 16 dims x 8 vectors
//   P              exp2(S c - base), fp16, transposed by movmatrix into a B operand
//   O^T += V^T P^T A = V^T: 16 dims x 16 tokens from two tokens' nibbles per
//                  byte times the two tokens' scales
//
// Rows of dims and tokens are numbered within the MMAs so that a lane's codes are
// contiguous (16 bytes of K, 8 or 16 of V), and the 16-byte pieces of a row are
// swizzled in shared memory so that both reads are free of bank conflicts.
// The base of a vector moves only when a logit comes near fp16's end above it (kHeadroom);
// sums are fp32 per lane and joined at the end.
//
// Measured (GB300): 4 requests of 131072 tokens, 32 heads on 4 of 128 (302 MB): 58.4 us,
// 5.2 TB/s (0.77 of the measured copy rate); 8 requests of 9000 to 32768 (92 MB): 27.2 us,
// 3.4 TB/s; one row over 4096 tokens: 9.7 us.  In the loop over chunks the copies run at
// 0.95 of the copy rate in the long case and 0.89 in the batched one; the rest is each part's
// start (division of the work 0.7 us, lookup and first pages 1.4 to 2.9), the join of the
// warps' states (1.3) and of a divided unit's records (1.3, to 5 in the CTA that joins), and
// the launch.  The other shapes (8 requests of 16384 tokens, 75 MB, floor 11.3 us): 16 vectors
// on 4 KV heads of 128 30.0 us, 8 on 2 of 256 24.1, 12 on 2 of 256 33.9 (a second tile of eight
// columns with half its products unused); 4 requests of 131072 tokens, 12 on 2 of 256, 81.5 us.
#include "qsa_dense_parts.cuh"

#include <algorithm>
#include <cmath>

namespace qsa {
namespace dense {
namespace {

// Bounds-check codes (reported by bounds-checked builds only).
[[maybe_unused]] constexpr int kChkChunk = 0x901;   // chunk: page id or token offset out of range
[[maybe_unused]] constexpr int kChkOut = 0x902;     // output row out of range
[[maybe_unused]] constexpr int kChkJoin = 0x903;    // descriptor, or the CTAs of a divided unit, out of range

// Four e2m1 pairs (bytes of w) -> four fp16 pairs.
__device__ __forceinline__ void e2m1x8(uint32_t w, uint32_t (&o)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
      : "r"(w));
}

__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 r;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a));
  return r;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint16_t r;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(r) : "r"(a));
  return r;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
  uint32_t r;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(r) : "r"(a));
  return r;
}

// D dims, NT tiles of 8 query vectors, W warps with S chunk buffers of TOK tokens.
template <int D_, int NT_, int W_, int S_, int TOK_>
struct Cfg {
  static constexpr int D = D_, NT = NT_, W = W_, S = S_, TOK = TOK_;
  static constexpr int kCols = NT * 8;
  static constexpr int kThreads = W * 32;
  static constexpr int kRow = D / 2;                 // code bytes of a token
  static constexpr int kSf = D / 16;                 // scale bytes of a token
  static constexpr int kK = TOK * kRow, kSc = TOK * kSf;
  static constexpr int kStage = 2 * kK + 2 * kSc;
  static constexpr int kRing = W * S * kStage;
  static constexpr int kJoin = W * kCols * (D + 2) * 4;   // the warps' states, over the ring
  static constexpr int kMain = kRing > kJoin ? kRing : kJoin;
  static constexpr int kQ = kCols * D * 2;           // queries in fragment order
  static constexpr int kMisc = kCols * 4 * 3;
  static constexpr int kSmem = kMain + kQ + kMisc;
  static constexpr int MT = TOK / 16;                // token tiles of a chunk
  static constexpr int KS = D / 16;                  // dim steps of S
  static constexpr int DT = D / 16;                  // dim tiles of O
};

// kRows: more than one row of each request, so that not all vectors see the same tokens.
template <class C, bool kRows>
__global__ void __launch_bounds__(C::kThreads, 1)
dense_decode_kernel(const __grid_constant__ Shape sh, const __grid_constant__ Work p) {
  constexpr int D = C::D, NT = C::NT, W = C::W, S = C::S, TOK = C::TOK;
  constexpr int MT = C::MT, KS = C::KS, DT = C::DT, kCols = C::kCols;
  extern __shared__ __align__(128) uint8_t smem[];
  const Geom& g = sh.g;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gid = lane >> 2, tig = lane & 3;
  uint4* s_q = reinterpret_cast<uint4*>(smem + C::kMain);        // [NT][KS / 2][32]
  float* s_cq = reinterpret_cast<float*>(smem + C::kMain + C::kQ);
  int* s_n = reinterpret_cast<int*>(s_cq + kCols);
  int* s_lo = s_n + kCols;

  pdl_wait();
  const Span span = plan_span<C::kThreads>(sh, p.seqlens, blockIdx.x, gridDim.x);
  pdl_trigger();
  if (span.begin >= span.end) return;

  // Token row within an 8-token group, by MMA row: see the swizzle below.
  constexpr uint32_t kPi = D == 128 ? 0x67542310u : 0x37156240u;
  auto pi = [&](int r) { return (int)((kPi >> (4 * r)) & 7u); };
  auto swz = [&](int t, int c) { return D == 128 ? c ^ ((t >> 1) & 3) : c ^ (t & 7); };
  // 16-byte pieces of the lane: K (row gid, pieces tig and, at D = 256, tig + 4), V (rows
  // 2 tig and 2 tig + 1; the dims that MMA row gid stands for)
  const int kr = pi(gid), v0r = pi(2 * tig), v1r = pi(2 * tig + 1);
  const uint32_t ring = smem_u32(smem) + warp * (S * C::kStage);
  const uint32_t k_off = kr * C::kRow + swz(kr, tig) * 16;
  const uint32_t k_off2 = kr * C::kRow + swz(kr, tig + 4) * 16;   // D = 256
  const uint32_t ks_off = 2 * C::kK + kr * C::kSf + 2 * tig;
  uint32_t v_off0, v_off1;
  if (D == 128) {
    v_off0 = C::kK + v0r * C::kRow + swz(v0r, gid >> 1) * 16 + (gid & 1) * 8;
    v_off1 = C::kK + v1r * C::kRow + swz(v1r, gid >> 1) * 16 + (gid & 1) * 8;
  } else {
    v_off0 = C::kK + v0r * C::kRow + swz(v0r, gid) * 16;
    v_off1 = C::kK + v1r * C::kRow + swz(v1r, gid) * 16;
  }
  const uint32_t vs_off0 = 2 * C::kK + C::kSc + v0r * C::kSf + gid * (D / 128);
  const uint32_t vs_off1 = 2 * C::kK + C::kSc + v1r * C::kSf + gid * (D / 128);
  // where this lane's copies of a chunk land: piece lane + 32 i of K and V
  constexpr int kPr = C::kRow / 16;                   // pieces of a row
  constexpr int kCopies = C::kK / 512;
  const uint32_t c_dst = (lane / kPr) * C::kRow + swz(lane / kPr, lane % kPr) * 16;
  static_assert(32 / kPr * kCopies == TOK, "copies");
  // (D = 256: four rows per copy, so every other one is four rows on in the swizzle)
  auto c_to = [&](int i) { return (D == 256 && (i & 1) ? c_dst ^ 64u : c_dst) + 512u * i; };

  const int psh = 31 - __clz(g.P);                   // log2 of the page size
  Cursor cursor(span);
  Seg seg;
  while (cursor.next(sh, p.seqlens, seg)) {
    // ---- the unit and this CTA's chunks of it ---------------------------------
    const int b = seg.b, kvh = seg.kvh, L = seg.L, todo = seg.todo, chunk0 = seg.chunk0;
    const int vec0 = seg.vec0, vecs = seg.vecs, cap = g.MB * g.P;
    const int n_all = seg.n_all, n_least = seg.n_least, lo_all = seg.lo_all, lo_most = seg.lo_most;
    const int mine = todo > warp ? (todo - warp + W - 1) / W : 0;   // this warp's chunks
    const bool partly = kRows && (n_least < n_all || lo_all < lo_most);   // not all vectors see the same

    // ---- the warp's query vectors: on their way while the pages are looked up ----------
    constexpr int kPer = (kCols + W - 1) / W, E = D / 32;
    uint2 raw[kPer][E / 4];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int c = warp + i * W;
      const bool real = c < vecs;
      const int j = real ? row_of(sh, vec0 + c) : 0, hh = real ? vec0 + c - j * sh.G : 0;
      const size_t row = ((size_t)b * g.R + j) * g.Hq + (size_t)kvh * sh.G + hh;
#pragma unroll
      for (int u = 0; u < E / 4; ++u)
        raw[i][u] = real ? *reinterpret_cast<const uint2*>(p.q + row * D + E * lane + 4 * u)
                         : make_uint2(0u, 0u);
    }
    // ---- page ids and copies ---------------------------------------------------
    int pages = -1;          // lane i: the page of this warp's chunk k, k % 32 = i
    uint32_t live = 0u;      // bit k % 32: chunk k has a page and its copies are under way
    auto load_pages = [&](int k0) {
      const int k = k0 + lane;
      pages = -1;
      if (k < mine && n_all > lo_all) {
        const int beta = ((chunk0 + warp + k * W) * TOK) >> psh;
        if (QSA_IN_BOUNDS(beta < g.MB, kChkChunk)) pages = p.page_table[(size_t)b * g.MB + beta];
        if (pages < 0 || pages >= g.NP) pages = -1;
      }
    };
    auto issue = [&](int k) {
      if ((k & 31) == 0 && k < mine) load_pages(k);
      const int page = __shfl_sync(0xffffffffu, pages, k & 31);
      const bool ok = k < mine && page >= 0 &&
                      QSA_IN_BOUNDS((((chunk0 + warp + k * W) * TOK) & (g.P - 1)) + TOK <= g.P &&
                                        kvh < g.Hkv && b < g.B, kChkChunk);
      live = (live & ~(1u << (k & 31))) | ((uint32_t)ok << (k & 31));
      if (ok) {
        const int tok = (chunk0 + warp + k * W) * TOK;
        const size_t row = (((size_t)page * g.Hkv + kvh) << psh) + (tok & (g.P - 1));
        const uint32_t st = ring + (k % S) * C::kStage;
        const uint8_t* kc = p.k_pool + row * C::kRow + lane * 16;
        const uint8_t* vc = p.v_pool + row * C::kRow + lane * 16;
#pragma unroll
        for (int i = 0; i < kCopies; ++i) cp_async16(st + c_to(i), kc + 512 * i);
#pragma unroll
        for (int i = 0; i < kCopies; ++i) cp_async16(st + C::kK + c_to(i), vc + 512 * i);
        const uint8_t* ksf = p.k_sf + row * C::kSf;
        const uint8_t* vsf = p.v_sf + row * C::kSf;
        if (C::kSc == 512) {
          cp_async16(st + 2 * C::kK + 16 * lane, ksf + 16 * lane);
          cp_async16(st + 2 * C::kK + 512 + 16 * lane, vsf + 16 * lane);
        } else {   // 256 bytes each: half a warp
          cp_async16(st + 2 * C::kK + 16 * lane, lane < 16 ? ksf + 16 * lane : vsf + 16 * lane - 256);
        }
      }
      cp_async_commit();
    };
#pragma unroll
    for (int k = 0; k < S - 1; ++k) issue(k);

    // ---- queries: fp16, scaled by a power of two into [256, 512), in the order of
    // the lanes that use them: dims 32 tig + 4 s.. of lane (gid, tig), step s ------
#pragma unroll
    for (int n = 0; n < kPer; ++n) {
      const int c = warp + n * W;
      if (kCols % W != 0 && c >= kCols) break;
      const bool real = c < vecs;
      const int j = real ? row_of(sh, vec0 + c) : 0;
      float x[E];
#pragma unroll
      for (int u = 0; u < E / 4; ++u) {
        x[4 * u] = __uint_as_float(raw[n][u].x << 16);
        x[4 * u + 1] = __uint_as_float(raw[n][u].x & 0xFFFF0000u);
        x[4 * u + 2] = __uint_as_float(raw[n][u].y << 16);
        x[4 * u + 3] = __uint_as_float(raw[n][u].y & 0xFFFF0000u);
      }
      float amax = 0.f;
#pragma unroll
      for (int i = 0; i < E; ++i) amax = fmaxf(amax, fabsf(x[i]));
#pragma unroll
      for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      const int ebits = (int)((__float_as_uint(amax) >> 23) & 0xFF);
      int sq = (amax > 0.f) ? 135 - ebits : 0;
      sq = sq > 126 ? 126 : (sq < -126 ? -126 : sq);
      const float up = __uint_as_float((uint32_t)(sq + 127) << 23);
      // dims d..d+3 are step s = (d % 32) / 4 of lane (c % 8, (d / 32) % 4), of the upper
      // eight steps past dim 128
#pragma unroll
      for (int u = 0; u < E / 4; ++u) {
        const int d = E * lane + 4 * u;
        const int st = ((d & 31) >> 2) + 8 * (d >> 7), to = (c & 7) * 4 + ((d >> 5) & 3);
        uint2* dst = reinterpret_cast<uint2*>(s_q + ((c >> 3) * (KS / 2) + (st >> 1)) * 32 + to) + (st & 1);
        *dst = make_uint2(pack_half2(x[4 * u] * up, x[4 * u + 1] * up),
                          pack_half2(x[4 * u + 2] * up, x[4 * u + 3] * up));
      }
      if (lane == 0) {
        const int sees = real ? visible_tokens(L, g.R, j, cap) : 0;
        s_cq[c] = real ? logit_factor(p, sq) : 1.f;
        s_n[c] = sees;
        s_lo[c] = first_seen(sees, sh.window);
      }
    }
    __syncthreads();

    float o[DT][NT][4], base[NT][2], sum[NT][2], cq[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        base[t][e] = kNoBase;
        sum[t][e] = 0.f;
        cq[t][e] = s_cq[8 * t + 2 * tig + e];
      }
#pragma unroll
      for (int i = 0; i < DT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][t][e] = 0.f;
    }

    // ---- chunks --------------------------------------------------------------------
    for (int k = 0; k < mine; ++k) {
      cp_async_wait<S - 2>();
      __syncwarp();
      const uint32_t st = ring + (k % S) * C::kStage;
      const int tok0 = (chunk0 + warp + k * W) * TOK;
      if ((live >> (k & 31)) & 1u) {
        const bool edge = tok0 + TOK > n_least || tok0 < lo_most;
        if (tok0 + TOK > n_all || tok0 < lo_all) {
          // tokens that no vector sees: their scales may be anything; 0 keeps 0 x V at 0
          for (int t = lane; t < TOK; t += 32)
            if (tok0 + t >= n_all || tok0 + t < lo_all) {
              const uint32_t a = st + 2 * C::kK + C::kSc + t * C::kSf;
#pragma unroll
              for (int i = 0; i < C::kSf / 8; ++i)
                asm volatile("st.shared.v2.u32 [%0], {%1, %1};" ::"r"(a + 8 * i), "r"(0u) : "memory");
            }
          __syncwarp();
        }
        if (partly && edge) {
          // Tokens that some of the vectors see and others do not: a NaN among the scales of V goes to the outputs
          // of those that see it, and out of V, where it would reach all (0 x NaN).  (As in qsa_dense8.cu.)
          const uint32_t sv = st + 2 * C::kK + C::kSc;
          // (between lo_most and n_least all see them)
          auto scales = [&](auto&& each) {
#pragma unroll 1
            for (int side = 0; side < 2; ++side) {
              const int from = max((side ? n_least : lo_all) - tok0, 0), to = min((side ? n_all : lo_most) - tok0, TOK);
#pragma unroll 1
              for (int x = from * C::kSf + lane; x < to * C::kSf; x += 32) each(sv + x);
            }
          };
          bool odd = false;
          scales([&](uint32_t at) { odd |= (lds8(at) & 0x7Fu) == 0x7Fu; });
          if (__any_sync(0xffffffffu, odd)) {
#pragma unroll 1
            for (int r = 0; r < TOK; ++r) {
              const int tok = tok0 + r;
              if (tok >= lo_most && tok < n_least) continue;
#pragma unroll
              for (int h = 0; h < D / 128; ++h) {          // 16 dims: output tiles 8 h.. of rows gid and gid + 8
                if ((lds8(sv + r * C::kSf + gid * (D / 128) + h) & 0x7Fu) != 0x7Fu) continue;
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                  for (int e = 0; e < 2; ++e) {
                    const int c = 8 * t + 2 * tig + e;
                    if (tok >= s_n[c] || tok < s_lo[c]) continue;
#pragma unroll
                    for (int i = 8 * h; i < 8 * h + 8; ++i)
                      o[i][t][e] = o[i][t][2 + e] = __uint_as_float(0x7FC00000u);
                  }
              }
            }
            __syncwarp();
            scales([&](uint32_t at) {
              if ((lds8(at) & 0x7Fu) == 0x7Fu) asm volatile("st.shared.u8 [%0], %1;" ::"r"(at), "h"((uint16_t)0) : "memory");
            });
            __syncwarp();
          }
        }
        // S^T
        float z[MT][NT][4];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) z[m][t][e] = 0.f;
#pragma unroll
          for (int hlf = 0; hlf < D / 128; ++hlf) {
            const uint32_t ko = hlf ? k_off2 : k_off;
            const uint4 wa = lds128(st + ko + (2 * m) * 8 * C::kRow);
            const uint4 wb = lds128(st + ko + (2 * m + 1) * 8 * C::kRow);
            const uint32_t sa = e4m3x2_to_f16x2(lds16(st + ks_off + 8 * hlf + (2 * m) * 8 * C::kSf));
            const uint32_t sb = e4m3x2_to_f16x2(lds16(st + ks_off + 8 * hlf + (2 * m + 1) * 8 * C::kSf));
            const uint32_t xa[4] = {wa.x, wa.y, wa.z, wa.w}, xb[4] = {wb.x, wb.y, wb.z, wb.w};
            const uint32_t s_a[2] = {prmt(sa, 0, 0x1010), prmt(sa, 0, 0x3232)};
            const uint32_t s_b[2] = {prmt(sb, 0, 0x1010), prmt(sb, 0, 0x3232)};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              uint32_t fa[4], fb[4];
              e2m1x8(xa[w], fa);
              e2m1x8(xb[w], fb);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                fa[i] = hmul2_u32(fa[i], s_a[w >> 1]);
                fb[i] = hmul2_u32(fb[i], s_b[w >> 1]);
              }
#pragma unroll
              for (int t = 0; t < NT; ++t) {
                const uint4 q = s_q[(t * (KS / 2) + 4 * hlf + w) * 32 + lane];
                const uint32_t a0[4] = {fa[0], fb[0], fa[1], fb[1]};
                const uint32_t a1[4] = {fa[2], fb[2], fa[3], fb[3]};
                mma_f16_16816(z[m][t], a0, q.x, q.y);
                mma_f16_16816(z[m][t], a1, q.z, q.w);
              }
            }
          }
        }
        if (edge) {
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int n = s_n[8 * t + 2 * tig + e], lo = s_lo[8 * t + 2 * tig + e];
#pragma unroll
              for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                  const int tok = tok0 + 16 * m + 8 * hf + kr;
                  if (tok >= n || tok < lo) z[m][t][2 * hf + e] = -INFINITY;
                }
            }
        }
        // the base: moved when a logit is far above it
        float top[NT][2];
        bool over = false;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = z[0][t][e];
#pragma unroll
            for (int m = 0; m < MT; ++m) x = fmaxf(x, fmaxf(z[m][t][e], z[m][t][2 + e]));
            top[t][e] = x * cq[t][e];
            over |= top[t][e] > base[t][e] + kHeadroom;
          }
        if (__any_sync(0xffffffffu, over)) {
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float x = top[t][e];
#pragma unroll
              for (int s2 = 4; s2 < 32; s2 <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, s2));
              const float nb = x > base[t][e] + kHeadroom ? x - kBelow : base[t][e];
              const float alpha = exp2_approx(base[t][e] - nb);
              base[t][e] = nb;
              sum[t][e] *= alpha;
#pragma unroll
              for (int i = 0; i < DT; ++i) {
                o[i][t][e] *= alpha;
                o[i][t][2 + e] *= alpha;
              }
            }
        }
        // P, then O^T
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          uint32_t pb[NT][2];
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const float p0 = exp2_approx(fmaf(z[m][t][2 * hf], cq[t][0], -base[t][0]));
              const float p1 = exp2_approx(fmaf(z[m][t][2 * hf + 1], cq[t][1], -base[t][1]));
              sum[t][0] += p0;
              sum[t][1] += p1;
              pb[t][hf] = movmatrix_trans(pack_weights(p0, p1));
            }
          uint32_t lo2[2][D / 64], hi2[2][D / 64], sc[2][D / 128];
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const uint32_t ro = (2 * m + hf) * 8 * C::kRow, so = (2 * m + hf) * 8 * C::kSf;
            uint32_t x0[D / 64], x1[D / 64];
            if constexpr (D == 128) {
              const uint2 u0 = lds64(st + v_off0 + ro), u1 = lds64(st + v_off1 + ro);
              x0[0] = u0.x; x0[1] = u0.y; x1[0] = u1.x; x1[1] = u1.y;
              sc[hf][0] = e4m3x2_to_f16x2(lds8(st + vs_off0 + so) | (lds8(st + vs_off1 + so) << 8));
            } else {
              const uint4 u0 = lds128(st + v_off0 + ro), u1 = lds128(st + v_off1 + ro);
              x0[0] = u0.x; x0[1] = u0.y; x0[2] = u0.z; x0[3] = u0.w;
              x1[0] = u1.x; x1[1] = u1.y; x1[2] = u1.z; x1[3] = u1.w;
              const uint32_t f0 = lds16(st + vs_off0 + so), f1 = lds16(st + vs_off1 + so);
              sc[hf][0] = e4m3x2_to_f16x2(prmt(f0, f1, 0x0040));
              sc[hf][1] = e4m3x2_to_f16x2(prmt(f0, f1, 0x0051));
            }
#pragma unroll
            for (int w = 0; w < D / 64; ++w) {
              lo2[hf][w] = (x0[w] & 0x0F0F0F0Fu) | ((x1[w] << 4) & 0xF0F0F0F0u);   // even dims
              hi2[hf][w] = ((x0[w] >> 4) & 0x0F0F0F0Fu) | (x1[w] & 0xF0F0F0F0u);   // odd dims
            }
          }
#pragma unroll
          for (int w = 0; w < D / 64; ++w) {
            uint32_t e0[4], d0[4], e1[4], d1[4];
            e2m1x8(lo2[0][w], e0);
            e2m1x8(hi2[0][w], d0);
            e2m1x8(lo2[1][w], e1);
            e2m1x8(hi2[1][w], d1);
            const uint32_t sx = sc[0][w >> 1], sy = sc[1][w >> 1];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t a[4] = {hmul2_u32(e0[i], sx), hmul2_u32(d0[i], sx),
                                     hmul2_u32(e1[i], sy), hmul2_u32(d1[i], sy)};
#pragma unroll
              for (int t = 0; t < NT; ++t) mma_f16_16816(o[4 * w + i][t], a, pb[t][0], pb[t][1]);
            }
          }
        }
      }
      __syncwarp();   // every lane has read this buffer before it is refilled
      issue(k + S - 1);
    }
    cp_async_wait<0>();
    __syncthreads();   // every warp's copies have landed and been read: the ring is free

    finish_unit<C, kChkOut, kChkJoin>(sh, p, span, cursor, seg, smem, s_n, o, base, sum,
                                      [](int gid, int i) { return (D / 8) * gid + 2 * i; });
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// The tile kernel's divided units joined: CTA (i, y, z) takes 32 vectors of the unit of
// descriptor i, a lane each (a record holds four dims of neighbouring vectors behind one
// another), its warps eight dims each.  The parts are added in their order.  The latency of the
// records is all there is, so up to three parts are asked for at once, their bases and sums with
// them (windowed verify rows over 8-bit pages 47.7 -> 45.3 us, 2 x 512 context rows 206.7 -> 202.0;
// with four or sixteen dims 45.6 and 45.4, 203.1 and 203.4), and eight of more.
// ---------------------------------------------------------------------------
constexpr int kJoinWarps = 8, kJoinQuads = 2;

template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32)
dense_join_kernel(const __grid_constant__ Shape sh, const __grid_constant__ Work p) {
  const Geom& g = sh.g;
  const int warp = blockIdx.z * kJoinWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  pdl_wait();
  pdl_trigger();
  const Desc d = p.desc[blockIdx.x];
  if (d.b < 0) return;
  // (a part whose waits gave up leaves no descriptor: what is there may be anything)
  if (!QSA_GUARD(d.b < g.B && d.tile >= 0 && d.tile < sh.tiles && d.kvh >= 0 && d.kvh < g.Hkv &&
                     d.first >= 0 && d.first < d.last && d.last < sh.ctas, kChkJoin))
    return;
  const int vec0 = d.tile * sh.vt, vecs = min(sh.vt, g.R * sh.G - vec0);
  const int c = blockIdx.y * 32 + lane;
  if (blockIdx.y * 32 >= vecs) return;
  const int parts = d.last - d.first + 1;
  const size_t rf = record_floats(sh.vt, D);
  auto record = [&](int i) {   // part i: slot 1 of the first CTA, slot 0 of the others
    return p.records + ((size_t)(d.first + i) * 2 + (i == 0 ? 1 : 0)) * rf;
  };
  if (c >= vecs) return;
  float m = kNoBase, l = 0.f;
  float4 acc[kJoinQuads];
#pragma unroll
  for (int q = 0; q < kJoinQuads; ++q) acc[q] = make_float4(0.f, 0.f, 0.f, 0.f);
  auto quad = [&](const float* rec, int q) {
    return reinterpret_cast<const float4*>(rec + 2 * sh.vt)[(size_t)(warp * kJoinQuads + q) * sh.vt + c];
  };
  auto add = [&](float mi, float li, const float4 (&x)[kJoinQuads]) {
    const float f = exp2_approx(mi - m);
    l = fmaf(li, f, l);
#pragma unroll
    for (int q = 0; q < kJoinQuads; ++q) {
      acc[q].x = fmaf(x[q].x, f, acc[q].x);
      acc[q].y = fmaf(x[q].y, f, acc[q].y);
      acc[q].z = fmaf(x[q].z, f, acc[q].z);
      acc[q].w = fmaf(x[q].w, f, acc[q].w);
    }
  };
  constexpr int kFew = 3;
  if (parts <= kFew) {           // (the usual: everything asked for at once)
    float mi[kFew], li[kFew];
    float4 x[kFew][kJoinQuads];
#pragma unroll
    for (int i = 0; i < kFew; ++i)
      if (i < parts) {
        const float* rec = record(i);
        mi[i] = rec[c];
        li[i] = rec[sh.vt + c];
#pragma unroll
        for (int q = 0; q < kJoinQuads; ++q) x[i][q] = quad(rec, q);
      }
#pragma unroll
    for (int i = 0; i < kFew; ++i)
      if (i < parts) m = fmaxf(m, mi[i]);
#pragma unroll
    for (int i = 0; i < kFew; ++i)
      if (i < parts) add(mi[i], li[i], x[i]);
  } else {
#pragma unroll 8
    for (int i = 0; i < parts; ++i) m = fmaxf(m, record(i)[c]);
#pragma unroll 8
    for (int i = 0; i < parts; ++i) {
      const float* rec = record(i);
      float4 x[kJoinQuads];
#pragma unroll
      for (int q = 0; q < kJoinQuads; ++q) x[q] = quad(rec, q);
      add(rec[c], rec[sh.vt + c], x);
    }
  }
  const int j = row_of(sh, vec0 + c), head = d.kvh * sh.G + (vec0 + c) - j * sh.G;
  const size_t row = ((size_t)d.b * g.R + j) * g.Hq + head;
  if (!QSA_IN_BOUNDS(j < g.R && head < g.Hq, kChkOut)) return;
  float f = 1.f;
  if (p.sinks) add_sink(p.sinks[head], m, l, f);
  const float r = l == 0.f ? 0.f : f * p.v_scale / l;
  uint2* to = reinterpret_cast<uint2*>(p.out + row * D) + warp * kJoinQuads;
#pragma unroll
  for (int q = 0; q < kJoinQuads; ++q) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(acc[q].x * r, acc[q].y * r);
    const __nv_bfloat162 hi = __floats2bfloat162_rn(acc[q].z * r, acc[q].w * r);
    to[q] = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  }
  if (warp == 0) p.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

}  // namespace
}  // namespace dense

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

size_t dense_carve(const dense::Shape& s, void* workspace, dense::Work* w) {
  size_t off = 256;
  uint8_t* base = reinterpret_cast<uint8_t*>(workspace);
  if (w) {
    w->status = reinterpret_cast<int*>(base);
    w->tickets = reinterpret_cast<int*>(base + off);
  }
  // (the same place for every geometry: a workspace may serve several, and tickets have to
  // be found at zero)
  off += ((size_t)sm_count() * sizeof(int) + 255) / 256 * 256;
  if (w) w->desc = reinterpret_cast<dense::Desc*>(base + off);
  off += ((size_t)dense::desc_count(s) * sizeof(dense::Desc) + 255) / 256 * 256;
  if (w) w->records = reinterpret_cast<float*>(base + off);
  off += (size_t)s.ctas * 2 * dense::record_floats(s.vt, s.g.D) * sizeof(float);
  return (off + 255) / 256 * 256;
}

cudaError_t launch_dense_join(const dense::Shape& s, const dense::Work& w, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(dense::desc_count(s), (std::min(s.vt, s.g.R * s.G) + 31) / 32,
                     s.g.D / (4 * dense::kJoinQuads * dense::kJoinWarps));
  cfg.blockDim = dim3(dense::kJoinWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto* kern = s.g.D == 256 ? dense::dense_join_kernel<256> : dense::dense_join_kernel<128>;
  return cudaLaunchKernelEx(&cfg, kern, s, w);
}

namespace {

using C128a = dense::Cfg<128, 1, 16, 3, 32>;
using C128b = dense::Cfg<128, 2, 8, 3, 64>;
using C256a = dense::Cfg<256, 1, 8, 3, 32>;
using C256b = dense::Cfg<256, 2, 8, 3, 32>;

// Query vectors per unit of the decode kernel: eight or sixteen (16384 tokens of 8 requests:
// eight vectors at head_dim 128 take 21.3 us in tiles of eight and 25.5 us in tiles of sixteen;
// sixteen vectors take 27.6 us in one tile, 33.4 us in two of eight).
int decode_cols(const Geom& g) { return g.R * (g.Hq / g.Hkv) <= 8 ? 8 : 16; }

dense::Shape decode_shape(const Geom& g, int window) {
  dense::Shape s;
  dense::set_heads(&s, g);
  s.vt = decode_cols(g);
  s.tiles = (g.R * s.G + s.vt - 1) / s.vt;
  const int tok = g.D == 256 ? 32 : (s.vt == 8 ? C128a::TOK : C128b::TOK);
  s.tok_sh = tok == 64 ? 6 : 5;
  s.window = window;
  s.least = 16;   // a chunk per warp (one row over 4096 tokens: 9.8, 9.7, 11.1 us with 8, 16, 32)
  // A part's start and end take what a CTA's warps take for three and a half chunks each
  // (16 warps: batched decode 27.9, 26.7, 25.3 and 25.8 us with 16, 32, 48 and 64, long
  // decode 61.3, 60.3, 59.0 and 57.6; 8 warps, 12 vectors of 256: 8 requests of up to 32768
  // tokens 44.8, 43.4, 42.0, 39.4, 39.9, 40.1 with 8, 12, 20, 28, 36 and 52, 4 of 131072 79.9,
  // 85.1, 82.2, 81.5, 80.7, 81.0; 16 vectors of 128: 32.4, 32.1, 30.7, 30.1, 30.7, 31.5).
  s.lead = 7 * (g.D == 128 && s.vt == 8 ? C128a::W : C128b::W) / 2;
  s.ctas = sm_count();
  s.by_unit = dense::unit_count(s) <= s.ctas;
  return s;
}

template <class C>
cudaError_t launch_decode(const dense::Shape& s, const dense::Work& w, cudaStream_t stream) {
  // (a single row has a kernel without what vectors that see different tokens need: batched decode 25.2 us, and
  // 26.1 with it)
  auto* kern = s.g.R > 1 ? dense::dense_decode_kernel<C, true> : dense::dense_decode_kernel<C, false>;
  static_assert(C::kSmem <= 227 * 1024, "shared memory");
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(s.ctas);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, s, w);
}

}  // namespace

// The tile kernel (128 to 512 query vectors per unit on tcgen05) takes more query vectors per
// KV head than one unit of the decode kernel's: with two units the cache is dequantised twice
// (16 requests of 16384 tokens, 32 vectors, tiles and two units: 64 us and 78 at head_dim 256;
// 48 vectors in three units 77 and 108 at 128, 65 and 108 at 256).  At head_dim 128 two units
// and tiles are alike up to 32 vectors: 76.8 us and 75.8 for that batch, 197.6 and 198.7 for 48
// requests, 57.5 and 61.0 for 64 of 2048 tokens, 25.3 and 27.8 for 32 in windows of 1024, but 17.4
// and 14.3 for two of 4096, 54.7 and 47.0 for one of 131072.  One rule for both head dims.
static bool use_tiles(const Geom& g) { return g.R * (g.Hq / g.Hkv) > 16; }

static dense::Shape dense_shape(const Geom& g, int window) {
  return use_tiles(g) ? dense_tile_shape(g, window) : decode_shape(g, window);
}

size_t dense_workspace_bytes(const Geom& g) {
  return dense_carve(dense_shape(g, 0), nullptr, nullptr);
}

cudaError_t launch_dense(const Geom& g, const DenseArgs& a, cudaStream_t stream) {
  const dense::Shape s = dense_shape(g, a.window);
  dense::Work w = {};
  w.q = reinterpret_cast<const __nv_bfloat16*>(a.q);
  w.k_pool = a.k_pool; w.k_sf = a.k_sf; w.v_pool = a.v_pool; w.v_sf = a.v_sf;
  w.v_scale = a.v_scale;
  w.z_mant = (float)frexp((double)a.k_scale * a.sm_scale * 1.4426950408889634, &w.z_exp);
  w.page_table = a.page_table; w.seqlens = a.seqlens;
  w.sinks = a.sinks;
  w.out = reinterpret_cast<__nv_bfloat16*>(a.out);
  w.lse = a.lse;
  dense_carve(s, a.workspace, &w);
  if (use_tiles(g)) {
    const cudaError_t e = launch_dense_tile(s, w, false, stream);
    return e != cudaSuccess ? e : launch_dense_join(s, w, stream);
  }
  if (g.D == 128)
    return s.vt == 8 ? launch_decode<C128a>(s, w, stream) : launch_decode<C128b>(s, w, stream);
  return s.vt == 8 ? launch_decode<C256a>(s, w, stream) : launch_decode<C256b>(s, w, stream);
}

}  // namespace qsa

QSA_BOUNDS_READER(bounds_word_dense)
