// qsa_dense8.cu -- dense attention over the 8-bit paged cache (e4m3 codes, a power
// of two for each 16 tokens and KV head), few query vectors per KV head: decode and
// narrow verify rows.
//
//   K = codes 2^ke, V = codes 2^ve,  ke and ve per block of 16 tokens
//   z_t = sm_scale q.K_t,  out = sum_t exp(z_t) V_t / sum_t exp(z_t)
//
// The division of the work, a warp's own stream of chunks and the joins are the NVFP4
// kernel's (qsa_dense.cu); the codes' part differs:
//
//   S^T = K Q^T    A = K: 16 tokens x 16 dims, e4m3 -> fp16 (exact; two codes an
//                  instruction, no product), B = Q.  A tile of 16 tokens is one block,
//                  so its scale is one factor of the tile's logits: c = cq 2^ke
//   P'             exp2(S c + ve - base): V's scale goes into the exponent, where it costs
//                  nothing, and O accumulates codes x P'.  The base follows the largest
//                  S c + ve.  Sums are of exp(z): a tile's P' times 2^-ve
//   O^T += V^T P'^T   A = V^T from two tokens' bytes, interleaved by one PRMT per two pairs
//
// Exponents lie at most 96 apart (bytes outside [95, 191] count as the nearest), and P' of the
// largest z + ve is at least 2^8 of fp32's normal range of 2^-126: a token whose V is as small
// as can be next to the largest still counts in the sum down to weights of 2^-38.
//
// Bound by the cache's bytes: 2 D + 1/8 per token and KV head.  Measured (GB300): 8 rows of 32 heads on 4
// of 128 over up to 32768 tokens each 33.6 us for 163 MB (floor 24.0), 16 of 8192 to 16384 38.8 us for 202 MB
// (5.2 TB/s, 0.77 of the copy rate; at 12 vectors a KV head 45.6); 24 on 2 of 256, 16 of these, 47.6; one
// row over 4096 tokens 9.8.  A warp's own chain (page, copy, S, weights, O) bounds it: the issue slots are
// 30 % busy, two warps to a scheduler; more warps with fewer tokens or stages each are slower (12 warps of
// 16 tokens 41.4 for 33.6), and so is turning codes to fp16 by their bits instead of conversions (39.4).
#include "qsa_dense_parts.cuh"

#include <cmath>

namespace qsa {
namespace dense {
namespace {

// Bounds-check codes (reported by bounds-checked builds only).
[[maybe_unused]] constexpr int kChkChunk = 0xC01;   // chunk: page id or token offset out of range
[[maybe_unused]] constexpr int kChkOut = 0xC02;     // output row out of range
[[maybe_unused]] constexpr int kChkJoin = 0xC03;    // the CTAs of a divided unit out of range

// D dims, NT tiles of 8 query vectors, W warps with S chunk buffers of TOK tokens.
template <int D_, int NT_, int W_, int S_, int TOK_>
struct Cfg8 {
  static constexpr int D = D_, NT = NT_, W = W_, S = S_, TOK = TOK_;
  static constexpr int kCols = NT * 8;
  static constexpr int kThreads = W * 32;
  static constexpr int kRow = D;                     // code bytes of a token
  static constexpr int kK = TOK * kRow;
  static constexpr int kStage = 2 * kK;
  static constexpr int kRing = W * S * kStage;
  static constexpr int kJoin = W * kCols * (D + 2) * 4;   // the warps' states, over the ring
  static constexpr int kMain = kRing > kJoin ? kRing : kJoin;
  static constexpr int kQ = kCols * D * 2;           // queries in fragment order
  static constexpr int kMisc = kCols * 4 * 3;
  static constexpr int kSmem = kMain + kQ + kMisc;
  static constexpr int MT = TOK / 16;                // token tiles (blocks) of a chunk
  static constexpr int KS = D / 16;                  // dim steps of S
  static constexpr int DT = D / 16;                  // dim tiles of O
  static_assert(MT == 1 || MT == 2, "a lane holds a chunk's exponents in a word");
};

// The exponents of a chunk's one or two blocks, as bytes within the append's range.
template <int MT>
__device__ __forceinline__ uint32_t load_exps(const uint8_t* p) {
  uint32_t x = MT == 2 ? *reinterpret_cast<const uint16_t*>(p) : *p;
  return __vminu4(__vmaxu4(x, 0x5F5F5F5Fu), 0xBFBFBFBFu);
}

// kRows: as in the NVFP4 kernel.
template <class C, bool kRows>
__global__ void __launch_bounds__(C::kThreads, 1)
dense8_decode_kernel(const __grid_constant__ Shape sh, const __grid_constant__ Work p) {
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

  // Token row within an 8-token group, by MMA row, and the place of a row's 16-byte piece:
  // the eight lanes that read together have K pieces tig of two rows four apart, or V pieces of
  // two dims' halves of four rows, all in different banks.
  constexpr uint32_t kPi = 0x37156240u;
  auto pi = [&](int r) { return (int)((kPi >> (4 * r)) & 7u); };
  auto swz = [&](int t, int c) { return c ^ (t & 7); };
  // K: row gid, pieces tig + 4 x (dims 64 x + 16 tig..); V: rows 2 tig and 2 tig + 1, pieces
  // gid + 8 x (dims 128 x + 16 gid..)
  const int kr = pi(gid), v0r = pi(2 * tig), v1r = pi(2 * tig + 1);
  const uint32_t ring = smem_u32(smem) + warp * (S * C::kStage);
  const uint32_t k_off = kr * C::kRow + swz(kr, tig) * 16;
  const uint32_t v_off0 = C::kK + v0r * C::kRow + swz(v0r, gid) * 16;
  const uint32_t v_off1 = C::kK + v1r * C::kRow + swz(v1r, gid) * 16;
  // where this lane's copies of a chunk land: piece lane + 32 i of K and V
  constexpr int kPr = C::kRow / 16;                   // pieces of a row
  constexpr int kCopies = C::kK / 512;
  const uint32_t c_dst = (lane / kPr) * C::kRow + swz(lane / kPr, lane % kPr) * 16;
  static_assert(32 / kPr * kCopies == TOK, "copies");
  // (32 / kPr rows per copy: that many rows on in the swizzle)
  auto c_to = [&](int i) { return (c_dst ^ (uint32_t)((((32 / kPr) * i) & 7) << 4)) + 512u * i; };

  // the dims of rows gid and gid + 8 of output tile i: this one and the next
  auto first_dim = [](int gid, int i) { return 128 * (i >> 3) + 16 * gid + 2 * (i & 7); };

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
    // ---- page ids, exponents and copies -----------------------------------------
    int pages = -1;          // lane i: the page of this warp's chunk k, k % 32 = i
    uint32_t exps_k = 0, exps_v = 0;     // and its blocks' exponents
    uint32_t now_k = 0, now_v = 0;       // of the 32 chunks that are being worked on
    uint32_t live = 0u;      // bit k % 32: chunk k has a page and its copies are under way
    auto load_pages = [&](int k0) {
      const int k = k0 + lane;
      pages = -1;
      if (k < mine && n_all > lo_all) {
        const int tok = (chunk0 + warp + k * W) * TOK, beta = tok >> psh;
        if (QSA_IN_BOUNDS(beta < g.MB, kChkChunk)) pages = p.page_table[(size_t)b * g.MB + beta];
        if (pages < 0 || pages >= g.NP) pages = -1;
        if (pages >= 0) {
          const size_t at = (((((size_t)pages * g.Hkv + kvh) << psh) + (tok & (g.P - 1)))) >> 4;
          exps_k = load_exps<MT>(p.k_sf + at);
          exps_v = load_exps<MT>(p.v_sf + at);
        }
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
      }
      cp_async_commit();
    };
#pragma unroll
    for (int k = 0; k < S - 1; ++k) issue(k);

    // ---- queries: fp16, scaled by a power of two into [256, 512), in the order of
    // the lanes that use them: dims 64 x + 16 tig + 4 s.. of lane (gid, tig), step 4 x + s ------
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
#pragma unroll
      for (int u = 0; u < E / 4; ++u) {
        const int d = E * lane + 4 * u;
        const int st = 4 * (d >> 6) + ((d >> 2) & 3), to = (c & 7) * 4 + ((d >> 4) & 3);
        uint2* dst = reinterpret_cast<uint2*>(s_q + ((c >> 3) * (KS / 2) + (st >> 1)) * 32 + to) + (st & 1);
        *dst = make_uint2(pack_half2(x[4 * u] * up, x[4 * u + 1] * up),
                          pack_half2(x[4 * u + 2] * up, x[4 * u + 3] * up));
      }
      if (lane == 0) {
        const int sees = real ? visible_tokens(L, g.R, j, cap) : 0;
        // (times a block's power of two it stays above zero and finite: a masked logit stays -inf)
        s_cq[c] = real ? fminf(fmaxf(logit_factor(p, sq), 0x1p-117f), 0x1p62f) : 1.f;
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
      if ((k & 31) == 0) {   // (these chunks' were loaded S - 1 chunks ago, the next ones' later)
        now_k = exps_k;
        now_v = exps_v;
      }
      const uint32_t ek = __shfl_sync(0xffffffffu, now_k, k & 31);
      const uint32_t ev = __shfl_sync(0xffffffffu, now_v, k & 31);
      cp_async_wait<S - 2>();
      __syncwarp();
      const uint32_t st = ring + (k % S) * C::kStage;
      const int tok0 = (chunk0 + warp + k * W) * TOK;
      if ((live >> (k & 31)) & 1u) {
        const bool edge = tok0 + TOK > n_least || tok0 < lo_most;
        if (tok0 + TOK > n_all || tok0 < lo_all) {
          // tokens that no vector sees: their codes may be NaN; 0 keeps 0 x V at 0
          for (int x = lane; x < TOK * kPr; x += 32) {
            const int tok = tok0 + x / kPr;
            if (tok >= n_all || tok < lo_all)
              asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(st + C::kK + 16 * x), "r"(0u)
                           : "memory");
          }
          __syncwarp();
        }
        if (partly && edge) {
          // Tokens that some of the vectors see and others do not: a NaN among their codes goes to the outputs
          // of those that see it, and out of V, where it would reach all (0 x NaN).  (Four rows of a window of 1024
          // 19.1 us without this, 19.5 so; 16 requests x 4 rows of 8192 to 16384 tokens 45.6 and 45.8.)
          const uint32_t sv = st + C::kK;
          // (the pieces x of these tokens; between lo_most and n_least all see them)
          auto pieces = [&](auto&& each) {
#pragma unroll 1
            for (int side = 0; side < 2; ++side) {
              const int from = max((side ? n_least : lo_all) - tok0, 0), to = min((side ? n_all : lo_most) - tok0, TOK);
#pragma unroll 1
              for (int x = from * kPr + lane; x < to * kPr; x += 32) each(x);
            }
          };
          uint32_t odd = 0u;
          pieces([&](int x) {
            const uint4 y = lds128(sv + 16 * x);
            odd |= nan_codes(y.x) | nan_codes(y.y) | nan_codes(y.z) | nan_codes(y.w);
          });
          if (__any_sync(0xffffffffu, odd != 0u)) {
#pragma unroll 1
            for (int r = 0; r < TOK; ++r) {
              const int tok = tok0 + r;
              if (tok >= lo_most && tok < n_least) continue;
#pragma unroll
              for (int i = 0; i < DT; ++i) {
                const int d = first_dim(gid, i);
                uint16_t two;
                asm volatile("ld.shared.u16 %0, [%1];" : "=h"(two) : "r"(sv + r * C::kRow + swz(r, d >> 4) * 16 + (d & 15)));
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                  for (int e = 0; e < 2; ++e) {
                    const int c = 8 * t + 2 * tig + e;
                    if (tok >= s_n[c] || tok < s_lo[c]) continue;
                    if ((two & 0x7F) == 0x7F) o[i][t][e] = __uint_as_float(0x7FC00000u);
                    if ((two & 0x7F00) == 0x7F00) o[i][t][2 + e] = __uint_as_float(0x7FC00000u);
                  }
              }
            }
            __syncwarp();
            pieces([&](int x) {
              const uint4 y = lds128(sv + 16 * x);
              asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(sv + 16 * x), "r"(without_nan(y.x)),
                           "r"(without_nan(y.y)), "r"(without_nan(y.z)), "r"(without_nan(y.w))
                           : "memory");
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
          for (int x = 0; x < D / 64; ++x) {
            // (piece tig + 4 x: the swizzle moves its lower three bits)
            const uint32_t ko = (k_off ^ (uint32_t)((x & 1) << 6)) + 128u * (x >> 1);
            const uint4 wa = lds128(st + ko + (2 * m) * 8 * C::kRow);
            const uint4 wb = lds128(st + ko + (2 * m + 1) * 8 * C::kRow);
            const uint32_t xa[4] = {wa.x, wa.y, wa.z, wa.w}, xb[4] = {wb.x, wb.y, wb.z, wb.w};
#pragma unroll
            for (int w = 0; w < 4; w += 2) {
              const uint32_t a0[4] = {e4m3x2_to_f16x2(xa[w] & 0xFFFFu), e4m3x2_to_f16x2(xb[w] & 0xFFFFu),
                                      e4m3x2_to_f16x2(xa[w] >> 16), e4m3x2_to_f16x2(xb[w] >> 16)};
              const uint32_t a1[4] = {e4m3x2_to_f16x2(xa[w + 1] & 0xFFFFu), e4m3x2_to_f16x2(xb[w + 1] & 0xFFFFu),
                                      e4m3x2_to_f16x2(xa[w + 1] >> 16), e4m3x2_to_f16x2(xb[w + 1] >> 16)};
#pragma unroll
              for (int t = 0; t < NT; ++t) {
                const uint4 q = s_q[(t * (KS / 2) + 2 * x + (w >> 1)) * 32 + lane];
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
        // a block's factor of its logits, and its exponent of V
        float c[MT][NT][2], ve[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const float two = __uint_as_float(((ek >> (8 * m)) & 0xFFu) << 23);
          ve[m] = (float)((int)((ev >> (8 * m)) & 0xFFu) - 127);
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              c[m][t][e] = cq[t][e] * two;
        }
        // the base: moved when a logit is far above it
        float top[NT][2];
        bool over = false;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = -INFINITY;
#pragma unroll
            for (int m = 0; m < MT; ++m)
              x = fmaxf(x, fmaf(fmaxf(z[m][t][e], z[m][t][2 + e]), c[m][t][e], ve[m]));
            top[t][e] = x;
            over |= x > base[t][e] + kHeadroom;
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
        // P', then O^T
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          uint32_t pb[NT][2];
          const float back = __uint_as_float((254u - ((ev >> (8 * m)) & 0xFFu)) << 23);   // 2^-ve
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const float b0 = ve[m] - base[t][0], b1 = ve[m] - base[t][1];
            float p0[2], p1[2];
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              p0[hf] = exp2_approx(fmaf(z[m][t][2 * hf], c[m][t][0], b0));
              p1[hf] = exp2_approx(fmaf(z[m][t][2 * hf + 1], c[m][t][1], b1));
              pb[t][hf] = movmatrix_trans(pack_weights(p0[hf], p1[hf]));
            }
            sum[t][0] = fmaf(p0[0] + p0[1], back, sum[t][0]);
            sum[t][1] = fmaf(p1[0] + p1[1], back, sum[t][1]);
          }
#pragma unroll
          for (int x = 0; x < D / 128; ++x) {
            uint4 u[2][2];
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const uint32_t ro = (2 * m + hf) * 8 * C::kRow + 128 * x;
              u[hf][0] = lds128(st + v_off0 + ro);
              u[hf][1] = lds128(st + v_off1 + ro);
            }
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              auto word = [&](const uint4& v) { return w == 0 ? v.x : w == 1 ? v.y : w == 2 ? v.z : v.w; };
#pragma unroll
              for (int h = 0; h < 2; ++h) {     // dims 4 w + 2 h and the next, of tokens 2 tig and 2 tig + 1
                const uint32_t lo = prmt(word(u[0][0]), word(u[0][1]), h ? 0x7362 : 0x5140);
                const uint32_t hi = prmt(word(u[1][0]), word(u[1][1]), h ? 0x7362 : 0x5140);
                const uint32_t a[4] = {e4m3x2_to_f16x2(lo & 0xFFFFu), e4m3x2_to_f16x2(lo >> 16),
                                       e4m3x2_to_f16x2(hi & 0xFFFFu), e4m3x2_to_f16x2(hi >> 16)};
#pragma unroll
                for (int t = 0; t < NT; ++t)
                  mma_f16_16816(o[8 * x + 2 * w + h][t], a, pb[t][0], pb[t][1]);
              }
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
                                      first_dim);
    __syncthreads();
  }
}

using C128a = Cfg8<128, 1, 8, 3, 32>;
using C128b = Cfg8<128, 2, 8, 3, 32>;
using C256a = Cfg8<256, 1, 8, 3, 16>;
using C256b = Cfg8<256, 2, 8, 3, 16>;

template <class C>
cudaError_t launch_decode8(const Shape& s, const Work& w, cudaStream_t stream) {
  auto* kern = s.g.R > 1 ? dense8_decode_kernel<C, true> : dense8_decode_kernel<C, false>;
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

Shape decode8_shape(const Geom& g, int window) {
  Shape s;
  set_heads(&s, g);
  s.vt = g.R * s.G <= 8 ? 8 : 16;
  s.tiles = (g.R * s.G + s.vt - 1) / s.vt;
  s.tok_sh = g.D == 128 ? 5 : 4;
  s.window = window;
  s.least = 16;
  // A part's start and end take what this many chunks take (batched decode 34.5, 33.9, 33.4, 33.6 us with
  // 28, 40, 48 and 68; 12 vectors of 256, 8 requests of 16384 tokens 42.2, 39.5, 37.5, 37.9 with 28, 40,
  // 68 and 84).
  s.lead = g.D == 128 ? 48 : 68;
  s.ctas = sm_count();
  s.by_unit = unit_count(s) <= s.ctas;
  return s;
}

}  // namespace
}  // namespace dense

// Above 16 vectors per KV head the tile kernel, as over NVFP4 pages (see there).  16 requests of 8192 to
// 16384 tokens, tiles and units of 16 here: 24 and 32 vectors 76.6 and 74.6 us at head_dim 128, 65.1 and
// 73.3 at 256 (tiles since then 59), 48 76.4 and 104; units of 32 vectors at 128 65.4 us, but 19.5 for 15.2
// with one request of 2000 tokens and 113 at 48 vectors.
static bool use_tiles(const Geom& g) { return g.R * (g.Hq / g.Hkv) > 16; }

static dense::Shape dense8_shape(const Geom& g, int window) {
  return use_tiles(g) ? dense_tile_shape(g, window) : dense::decode8_shape(g, window);
}

size_t dense8_workspace_bytes(const Geom& g) {
  return dense_carve(dense8_shape(g, 0), nullptr, nullptr);
}

cudaError_t launch_dense8(const Geom& g, const DenseArgs& a, cudaStream_t stream) {
  const dense::Shape s = dense8_shape(g, a.window);
  dense::Work w = {};
  w.q = reinterpret_cast<const __nv_bfloat16*>(a.q);
  w.k_pool = a.k_pool; w.k_sf = a.k_sf; w.v_pool = a.v_pool; w.v_sf = a.v_sf;
  w.v_scale = 1.f;
  w.z_mant = (float)frexp((double)a.sm_scale * 1.4426950408889634, &w.z_exp);
  w.page_table = a.page_table; w.seqlens = a.seqlens;
  w.sinks = a.sinks;
  w.out = reinterpret_cast<__nv_bfloat16*>(a.out);
  w.lse = a.lse;
  dense_carve(s, a.workspace, &w);
  if (use_tiles(g)) {
    const cudaError_t e = launch_dense_tile(s, w, true, stream);
    return e != cudaSuccess ? e : launch_dense_join(s, w, stream);
  }
  if (g.D == 128)
    return s.vt == 8 ? dense::launch_decode8<dense::C128a>(s, w, stream)
                     : dense::launch_decode8<dense::C128b>(s, w, stream);
  return s.vt == 8 ? dense::launch_decode8<dense::C256a>(s, w, stream)
                   : dense::launch_decode8<dense::C256b>(s, w, stream);
}

}  // namespace qsa

QSA_BOUNDS_READER(bounds_word_dense8)
