// qsa_dense_tile.cu -- dense attention over the NVFP4 paged cache, or the 8-bit one
// (E8: see "8-bit pages"), for many query vectors per KV head (context row groups,
// wide verify rows), on the fifth-generation tensor cores.
//
// TensorRT-LLM PR #20276 ("Qwen3.8-Flash-Next NVFP4 target"), Performance:
// context rows run on tcgen05 with K/V tiles shared by a group of rows; Known
// limitations: context rows read the NVFP4 pages dequantised on the way.
//
// The work is 4 D flops per (query vector, token), on the tensor core:
//   S = Q K^T    A = Q, B = K from shared memory (K-major), D = S in tensor memory
//   O += P V     A = P from tensor memory, B = V from shared memory (token rows, MN-major)
// A tile is 128 query vectors (row, head) of one request and KV head: the 128
// tensor-memory lanes of a CTA.
//
// Pairs of CTAs (more than two tiles of vectors per KV head at head_dim 128,
// more than one at 256): the two SMs of a pair run M = 256 MMAs (cta_group::2)
// on two tiles at once, each SM holding half of every K and V tile (half the
// tokens of K, half the dims of V).  So each SM dequantises half of a chunk and
// feeds half of the B operand from its shared memory; with one SM per tile,
// operand reads and the dequantised stores fill shared memory's bandwidth and
// everything else that uses it (barrier probes) crawls (two context chunks of
// 1024 rows: 941 us, by pairs 811).  At head_dim 128 a CTA has two tiles (four
// per pair), at 256 one.  Single CTAs (fewer vectors, from 17 on: verify rows)
// have one tile, for which the cache's bytes, not the products, are the floor.
//
// Measured over NVFP4 pages (GB300, SM clock 2070 MHz):
//   two context chunks of 1024 rows, 32 heads on 4, behind 30000 tokens: 646 us,
//   1.57 PFLOP/s (0.81 of the measured cuBLAS rate).  The tensor pipe is active
//   70 % of the time: a chunk's turn takes 2940 cycles of which its MMAs need 2048,
//   the rest is the softmax's latency between a tile's turns.
//   The same at 24 heads on 2 of 256: 966 us, 1.68 PFLOP/s (0.85); 4 x 256 rows of
//   these over 16384 tokens 268 us (floor 208).
//   32 requests x 4 verify rows, 24 heads on 2, head_dim 256, window 4096: 41.5 us
//   for 79 MB (floor 11.8).  A CTA has 30 chunks of 64 tokens, 1780 cycles each (the K
//   warps' conversion, shared memory; the MMAs need 1024, 80 of the tile's 128 rows hold
//   no vector), a start of 5.6 us (work division 0.7,
//   queries 4.3, first pages and S 0.6), a record (1.2 us), and the join kernel with its
//   launch (5 to 6 us).  16 requests x 4 rows of 32 heads on 4 of 128 over 16384 tokens: 79 us
//   for 151 MB (floor 22.6).
//
// Roles in a CTA (a warp group each unless noted):
//   softmax   a thread per vector (tensor-memory lane): its row of S to registers, base
//             (moved only where a weight would overflow), P = exp2(S c - base) as
//             fp16 over the columns of S it has read, 64 tokens at a time, sums in fp32;
//             at the end of a part O from tensor memory to the output or to a record.  A
//             group per tile
//   copy      one warp: codes and scales of the pages by bulk copies some chunks ahead
//   dequant   e2m1 x e4m3 (8-bit pages: e4m3 alone) exact in fp16 into double-buffered K and V tiles
//             (128-byte swizzle)
//   inspector one warp (NVFP4 pages, two tiles): see "Values that are not finite"
//   MMA       one warp (of the pair's first CTA) issues every MMA in order.  With two tiles
//             they take turns: O_0, S_0 of the next chunk, O_1, S_1, so that one tile's
//             softmax runs under the other's products; with one, S has two buffers
//             and runs two chunks ahead.  (A warp per tile, whose MMAs on two accumulators
//             interleave, took twice the time: runs of MMAs on one accumulator are what
//             the tensor core pipelines.)
// P lies over S: S of the next chunk is issued behind the O that reads P, and
// MMAs of one thread run in order, so no barrier guards the reuse.
//
// Tensor memory (512 columns): the two S buffers from column 0, O from 256, and with one
// tile Q (384 at head_dim 128, 128 at 256).
// mbarriers, all waits bounded (2 s; a wait that gives up sets the status word).
// Arrivals are one per warp; those for the MMA warp go to the first CTA's barrier,
// commits to both CTAs':
//   qready        Q tiles written; O, S of the part before read    (softmax warps)
//   full[i]       stage i of codes and scales there                (bulk copies)
//   empty[i]      stage i read                                     (the converting warps, the inspector)
//   kready/vready[x]  K / V tile x written                         (its four converting warps)
//   kfree/vfree[x]    MMAs that read tile x complete               (commit)
//   barS[y]       S buffer y complete -- and, with two tiles, every MMA before it,
//                 so also the tile's O so far; once more after a part's last O   (commit)
//   barO          O complete up to a chunk (one tile)              (commit)
//   partO         O complete at the end of a part (one tile)       (commit)
// A phase of a barrier is only told from its neighbours, so every waiter is at most
// one phase behind: barO is waited for only where barS has said that the phase
// before is complete, and the part's end has a barrier of its own.
//   pready[y][h]  half h of P in buffer y written                  (four softmax warps)
#include "qsa_dense.cuh"
#include "qsa_tc_pair.cuh"

#include <type_traits>

namespace qsa {
namespace dense {
namespace {

using namespace tc;

// Bounds-check codes (reported by bounds-checked builds only).
[[maybe_unused]] constexpr int kChkChunk = 0xA01;   // copy: token offset or place in the ring out of range
[[maybe_unused]] constexpr int kChkOut = 0xA02;     // output row out of range
[[maybe_unused]] constexpr int kChkRecord = 0xA03;  // record's slot out of range

// In `copied`: the chunk has tokens that some vectors see and others do not (see "Values that are not finite").
constexpr uint32_t kMarked = 0x80000000u;

// E8: the 8-bit cache's pages instead of NVFP4's (see "8-bit pages" below).
template <int D_, int CG_, bool E8_>
struct TT {
  static constexpr int D = D_, CG = CG_;                 // CG: CTAs per MMA
  static constexpr bool E8 = E8_;
  static constexpr bool kInspect = !E8 && D == 128 && CG == 2;   // (an inspector: see "Values that are not finite")
  static constexpr int kTiles = D == 128 && CG == 2 ? 2 : 1;   // tiles of a CTA
  static constexpr int kTok = D == 256 ? 64 : 128;       // tokens per chunk
  static constexpr int kHalves = kTok / 64;              // P is written 64 tokens at a time
  static constexpr int kSoft = 4 * kTiles;               // softmax warps
  // Dequantisation warps: four K and four V, or, where a CTA has half of every tile and
  // two softmax groups, four that convert both.
  static constexpr int kDeq = kTiles == 2 ? 4 : 8;
  static constexpr int kMma = kSoft + kDeq;              // the MMA warp; its group's others idle
  static constexpr int kThreads = 32 * (kMma + 4);
  // Registers per thread after the roles part (128 at launch): the softmax holds a
  // row's 128 logits.
  static constexpr int kSoftRegs = 192;
  static constexpr int kDeqRegs = kTiles == 2 ? 72 : 96;
  static constexpr int kMmaRegs = kTiles == 2 ? 56 : 72;
  static_assert(32 * (kSoft * kSoftRegs + kDeq * kDeqRegs + 4 * kMmaRegs) <= kThreads * 128 &&
                    kThreads == 512, "registers");
  static constexpr int kVecs = 128 * CG * kTiles;        // query vectors of a unit
  static constexpr int kKRows = kTok / CG;               // K tile: tokens of this CTA
  static constexpr int kKBlk = kKRows * 128;             // its 64-dim blocks
  static constexpr int kKBytes = kKRows * D * 2;
  static constexpr int kVDims = D / CG;                  // V tile: dims of this CTA
  static constexpr int kVBlk = kTok * 128;
  static constexpr int kVBytes = kTok * kVDims * 2;
  // Tensor-memory columns of O and of Q, which leaves shared memory's bandwidth to K and
  // V; with two tiles there is no room and Q stays in shared memory.
  static constexpr uint32_t kOCol = 256;
  static constexpr bool kQTmem = kTiles == 1;
  static constexpr uint32_t kQCol = D == 128 ? 384 : 128;
  static_assert(kQCol + D / 2 <= 512 && 2 * kTok <= 256, "tensor-memory columns");
  // Q tiles (D/64 blocks of 128 rows x 128 B), or, with Q in tensor memory, 8 KB per warp
  // through which Q and O pass.
  // Single CTAs over 8-bit pages at head_dim 256 leave that out (a thread reads its row of Q by itself,
  // rows of O are transposed between four lanes) for a third stage, as their copies' latency bounds
  // them: 48 vectors a KV head, 16 requests of 8192 to 16384 tokens, 66.3 us before, 59.0 now, windowed
  // verify rows 52.9 and 47.8.  (At head_dim 128 the softmax does: 76.7 and 77.2; pages asked for in L2
  // ahead of their copies, 63.3 with two stages, 59.7 with three.)
  static constexpr bool kPass = !(E8 && CG == 1 && D == 256);
  static constexpr int kQBytes = !kPass ? 0 : kQTmem ? 32768 : 128 * D * 2;
  // Codes and scales on their way: a stage is a chunk, this CTA's K rows and whole V rows.
  static constexpr int kDepth = CG == 2 ? 4 : E8 && kPass ? 2 : 3;   // (what there is room for)
  static constexpr int kRow = E8 ? D : D / 2;            // code bytes of a token
  static constexpr int kKCodes = kKRows * kRow, kVCodes = kTok * kRow;
  static constexpr int kKPart = kKCodes + (E8 ? 0 : kKCodes / 8), kVPart = kVCodes + (E8 ? 0 : kVCodes / 8);
  static constexpr int kStage = kKPart + kVPart;
  static constexpr int kRing = kDepth * kStage;
  static constexpr int kBars = 18 + 2 * kDepth;
  // Scales of a chunk's blocks, in a ring of their own: eight floats 2^ke, ve and 2^-ve each.
  static constexpr int kExpSlots = E8 ? 8 : 0, kExpFloats = 24;
  static_assert(!E8 || kExpSlots >= kDepth + 2, "exponents' ring");
  static constexpr int kSmem = 1024 + kTiles * kQBytes + 2 * kKBytes + 2 * kVBytes + kRing +
                               kBars * 8 + 16 + (E8 ? 16 : kDepth * 20 + 4) + kExpSlots * kExpFloats * 4;
  static_assert(kVecs <= 512 && (!E8 || kDepth <= 4), "a unit's vectors; what is copied of each stage");
};

// Asynchronous copy of 16 bytes, zeros where `on` is false.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// ---- values that are not finite ----------------------------------------------------
// A weight of 0 times a V that is not finite is NaN: of a token that some of the unit's vectors see and others
// do not, such a value would reach the others.  The converters leave these values out of the tile and leave a note
// (in a pair, whose converters have half of the dims each, in both CTAs) ahead of the arrival that lets the MMAs
// begin.  Where there is one, the CTA goes through all its parts once more when everything is done, and vectors
// get what was left out from the pages themselves.  (Given to the vectors by the softmax warps at the end of each part
// it cost them registers: 2 x 512 context rows over 8-bit pages 207 -> 210 us, by a function that these call 240.)
// 8-bit pages: looked for in the tiles as stored.  (2 x 512 context rows, 24 vectors of 128, windowed verify, 4 x 256
// rows of 256: without any of it 203.5, 76.8, 45.4 and 313 us; so 207, 78.4, 45.5 and 307; in the codes' registers
// 209, 84, 46.0 and 308.)
// NVFP4 pages: in the scales of the stages that the copy warp marks as having such tokens, which the same lane
// reads next.  Where four warps convert both K and V they have no registers left for it (two context chunks 656 us),
// and a warp of its own, the inspector, does it, which they wait for at marked stages (646; 637 without; with an
// inspector for all, 16 requests x 4 rows of 32 heads on 4 of 128 86 us instead of 79, windowed verify 41.8 for 41.5).
__device__ __forceinline__ bool partly_seen(const Seg& seg, int tok) {
  return tok < seg.n_all && tok >= seg.lo_all && (tok >= seg.n_least || tok < seg.lo_most);
}
// Whether the `tokens` from tok0 on can have such tokens.
__device__ __forceinline__ bool any_partly(const Seg& seg, int tok0, int tokens) {
  return (seg.n_least < seg.n_all && tok0 + tokens > seg.n_least) || (seg.lo_all < seg.lo_most && tok0 < seg.lo_most);
}
// Bits 15 and 31 for two fp16 that are not finite (the others are anything), and those as zeros.
__device__ __forceinline__ uint32_t not_finite2(uint32_t w) { return (w & 0x7C007C00u) + 0x04000400u; }
__device__ __forceinline__ uint32_t finite2(uint32_t w) {
  return w & ~(((not_finite2(w) & 0x80008000u) >> 15) * 0xFFFFu);
}
template <int CG>
__device__ __forceinline__ void leave_note(uint32_t* at) {
  if constexpr (CG == 1)
    *reinterpret_cast<volatile uint32_t*>(at) = 1u;
  else
    asm volatile(
        "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, 0;\n\tst.shared::cluster.u32 [a], %1;\n\t"
        "mapa.shared::cluster.u32 a, %0, 1;\n\tst.shared::cluster.u32 [a], %1;\n\tfence.acq_rel.cluster;\n\t}" ::"r"(
            smem_u32(at)), "r"(1u)
        : "memory");
}

// ---- copies ----------------------------------------------------------------------
// The copy warp brings every chunk's codes and scales into the ring, kDepth chunks ahead
// (copies by the converting warps themselves took a third of their time: windowed verify
// rows 50 -> 46 us without, two context chunks 673 -> 648):
// a piece of a page (as many rows as the chunk has of it) is contiguous, so that a chunk is
// at most eight bulk copies, one per lane.  Pages that are not there, and pieces that no row
// of the unit sees, are not copied; `copied` says so (bit per lane of the stage's copies).
template <class T>
__device__ __forceinline__ bool copy_all(const Shape& sh, const Work& p, const Span& span, int rank,
                                         uint8_t* ring, uint64_t* full, uint64_t* empty,
                                         volatile uint32_t* copied, float* exps, int* sides) {
  const int lane = threadIdx.x & 31;
  const int psh = 31 - __clz(sh.g.P);
  const bool scales = lane & 1, v = lane & 2;         // (8-bit: no copies of scales)
  const int rows = v ? T::kTok : T::kKRows;
  const int step = min(sh.g.P, rows);                 // rows of a copy
  const int off = (lane >> 2) * step;                 // its first, in the stage's part
  const bool mine = lane < 8 && off < rows && !(T::E8 && scales);
  const int tok_off = off + (v ? 0 : rank * T::kKRows);
  const uint32_t row_bytes = scales ? T::D / 16 : T::kRow, bytes = step * row_bytes;
  const uint8_t* pool = v ? (scales ? p.v_sf : p.v_pool) : (scales ? p.k_sf : p.k_pool);
  uint8_t* dst = ring + (v ? T::kKPart + (scales ? T::kVCodes : 0) : (scales ? T::kKCodes : 0)) +
                 off * row_bytes;
  const uint64_t policy = policy_evict_normal();   // (other units read the page too)
  int slot = 0, use = 0;
  [[maybe_unused]] int chunks = 0;
  bool ok = true;
  Cursor cursor(span);
  Seg seg;
  while (ok && cursor.next(sh, p.seqlens, seg)) {
    // page ids: lane i has that of block blk0 + i, and `later` of blk0 + 32 + i
    auto page_id = [&](int beta) {
      return beta < sh.g.MB && seg.n_all > seg.lo_all
                 ? __ldg(p.page_table + (size_t)seg.b * sh.g.MB + beta) : -1;
    };
    int blk0 = (seg.chunk0 * T::kTok) >> psh;
    int ids = page_id(blk0 + lane), later = page_id(blk0 + 32 + lane);
    // 8-bit: lane i has the exponent of block i & 7 of the chunk, of K (i < 8) or of V
    auto exp_of = [&](int tok0) {
      const int tok = tok0 + 16 * (lane & 7), at = (tok >> psh) - blk0;
      const int here = __shfl_sync(0xffffffffu, ids, at & 31);
      const int page_later = __shfl_sync(0xffffffffu, later, at & 31);
      const int page = at < 32 ? here : page_later;
      uint32_t e = 127u;
      if (lane < 16 && 16 * (lane & 7) < T::kTok && page >= 0 && page < sh.g.NP && tok < seg.n_all &&
          tok + 16 > seg.lo_all)
        e = __ldg((lane < 8 ? p.k_sf : p.v_sf) +
                  (((((size_t)page * sh.g.Hkv + seg.kvh) << psh) + (tok & (sh.g.P - 1))) >> 4));
      return e;
    };
    [[maybe_unused]] uint32_t exp_next = 0;
    if constexpr (T::E8) exp_next = exp_of(seg.chunk0 * T::kTok);
#pragma unroll 1
    for (int c = 0; c < seg.todo; ++c) {
      const int tok0 = (seg.chunk0 + c) * T::kTok, tok = tok0 + tok_off;
      if ((tok0 >> psh) - blk0 >= 32) {
        blk0 += 32;
        ids = later;
        later = page_id(blk0 + 32 + lane);
      }
      const int at = (tok >> psh) - blk0;             // (a chunk is four pages at most)
      const int here = __shfl_sync(0xffffffffu, ids, at & 31);
      const int page_later = __shfl_sync(0xffffffffu, later, at & 31);
      const int page = at < 32 ? here : page_later;
      const bool there =
          mine && page >= 0 && page < sh.g.NP && tok < seg.n_all && tok + step > seg.lo_all &&
          QSA_IN_BOUNDS(tok >= 0 && (tok & (sh.g.P - 1)) + step <= sh.g.P && slot < T::kDepth &&
                            off + step <= rows && seg.kvh < sh.g.Hkv && seg.b < sh.g.B && at < 64,
                        kChkChunk);
      const uint32_t which = __ballot_sync(0xffffffffu, there);
      const uint32_t sum = __reduce_add_sync(0xffffffffu, there ? bytes : 0u);
      if (use > 0 && gave_up(&empty[slot], use - 1)) { ok = false; break; }
      if constexpr (!T::E8) {
        if (lane == 0) {
          const bool marked = any_partly(seg, tok0, T::kTok);
          if (marked) {
            int* at_slot = sides + 4 * slot;
            at_slot[0] = seg.lo_all - tok0;
            at_slot[1] = seg.lo_most - tok0;
            at_slot[2] = seg.n_least - tok0;
            at_slot[3] = seg.n_all - tok0;
          }
          copied[slot] = which | (marked ? kMarked : 0u);
          mbar_arrive_expect_tx(&full[slot], sum);
        }
        __syncwarp();
      }
      if (there)
        bulk_g2s(dst + slot * T::kStage,
                 pool + ((((size_t)page * sh.g.Hkv + seg.kvh) << psh) + (tok & (sh.g.P - 1))) * row_bytes,
                 bytes, &full[slot], policy);
      if constexpr (T::E8) {
        // The exponents are written before the stage's one arrival (the copies' bytes may be
        // counted before they are expected: without the arrival the phase stays).  Their place
        // was last chunk - kExpSlots', which every softmax warp is done with: the stage was
        // free, so V of chunk - kDepth was converted, for which the MMAs that read the weights of
        // chunk - kDepth - 2 had completed.
        if (lane < 16) {
          const uint32_t e = min(max(exp_next, 95u), 191u);
          float* to = exps + T::kExpFloats * (chunks & (T::kExpSlots - 1)) + lane;
          *to = lane < 8 ? __uint_as_float(e << 23) : (float)((int)e - 127);
          if (lane >= 8) to[8] = __uint_as_float(0x7F000000u - (e << 23));
        }
        __syncwarp();
        if (lane == 0) {
          copied[slot] = which;
          mbar_arrive_expect_tx(&full[slot], sum);
        }
        ++chunks;
        if (c + 1 < seg.todo) exp_next = exp_of(tok0 + T::kTok);
      }
      if (++slot == T::kDepth) {
        slot = 0;
        ++use;
      }
    }
  }
  // Nothing may still be on its way when the block ends, whoever gave up: the last use
  // of each stage.
  for (int x = 0; x < T::kDepth; ++x) {
    const int uses = use + (x < slot ? 1 : 0);
    if (uses > 0 && gave_up(&full[x], uses - 1)) ok = false;
  }
  return ok;
}

// ---- dequantisation --------------------------------------------------------------
// A converter turns this CTA's part of every chunk's K (kKRows tokens, all dims) or V
// (all tokens, kVDims dims) into a tile, four warps with a 16-byte piece (32 codes,
// two scales) per lane and step.  Neighbouring lanes have neighbouring pieces, four of eight
// rows or two of sixteen; the eight lanes that store together would meet in two 64-dim
// blocks' same banks, so the upper two pieces of four go in another order.
//
// The code is kept small (one copy for K and V where the shapes agree, no
// unrolling over chunks): with four roles' loops on an SM, instruction-cache misses
// were its largest stall (windowed verify rows 85 -> 60 us by one copy instead of two).
template <class T, int kRows, int kDims>
struct Converter {
  static constexpr int D = T::D;
  static constexpr int kPieces = kDims / 32;                  // 16-byte pieces of a row
  static constexpr int kUnits = kRows * kPieces / 128;        // steps of a warp
  static constexpr int kBlk = kRows * 128, kBytes = kRows * kDims * 2;

  uint8_t* tiles;
  uint64_t *ready, *freed;
  uint32_t part;                 // the stage's part: codes, and behind them scales
  int row0, lane_sh;
  // Per step: row of the part, place in it and its scales' place, place in the tile.
  int row[kUnits];
  uint32_t at_c[kUnits], at_s[kUnits], at_t[kUnits];

  __device__ __forceinline__ Converter(const Shape& sh, bool v, int token0, int dim0, int dw, uint8_t* ring,
                                       uint8_t* tiles_, uint64_t* ready_, uint64_t* freed_)
      : tiles(tiles_), ready(ready_), freed(freed_), part(smem_u32(ring) + (v ? T::kKPart : 0)),
        row0(token0) {
    const int lane = threadIdx.x & 31;
    lane_sh = 31 - __clz(min(sh.g.P, kRows));                 // log2 of a copy's rows
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int u = dw + 4 * i;
      int r, piece;
      if (kPieces >= 4) {
        r = 8 * (u % (kRows / 8)) + (lane >> 2);
        piece = 4 * (u / (kRows / 8)) + (lane & 3);
      } else {
        r = 16 * u + (lane >> 1);
        piece = lane & 1;
      }
      row[i] = r;
      // eight dims 4 piece + u: block (4 piece) / 8, chunk 4 (piece & 1) + u, by xor
      at_t[i] = (piece >> 1) * kBlk + sw128(r, 4 * (piece & 1));
      at_c[i] = r * (D / 2) + dim0 / 2 + 16 * piece;
      at_s[i] = kRows * (D / 2) + r * (D / 16) + dim0 / 16 + 2 * piece;
    }
  }
  // Chunk number `chunks` of the CTA, from token tok0, out of stage `slot` into its tile; false
  // when the wait for the tile gave up.
  __device__ __forceinline__ bool convert(const Seg& seg, int tok0, int chunks, int slot, uint32_t copied,
                                          bool v, uint32_t* note) {
    const int lane = threadIdx.x & 31;
    const int x = chunks & 1, use = chunks >> 1;
    uint8_t* tile = tiles + x * kBytes;
    const uint32_t from = part + slot * T::kStage;
    const bool flip = kPieces >= 4 && (lane & 2);
    // Rows that no vector of the unit sees, and what was not copied, become zeros by their scales
    // (a code is always finite).
    const int first = seg.lo_all - tok0 - row0;
    const uint32_t seen = (uint32_t)max(seg.n_all - seg.lo_all, 0);
    const uint32_t bits = copied >> (v ? 2 : 0);
    if (!T::kInspect && v && (copied & kMarked)) {
      // NaN among the scales of tokens that some vectors see and others do not: zeros in the stage, where
      // this lane alone reads them
      const int* at_slot = reinterpret_cast<const int*>(note + 2 + T::kDepth) + 4 * slot;   // (behind `copied`)
      bool odd = false;
#pragma unroll 1
      for (int i = 0; i < kUnits; ++i) {
        const int u = ((threadIdx.x >> 5) & 3) + 4 * i;
        const int r = kPieces >= 4 ? 8 * (u % (kRows / 8)) + (lane >> 2) : 16 * u + (lane >> 1);
        const int up = kPieces >= 4 ? 4 * (u / (kRows / 8)) : 0;      // (pieces on from the first step's)
        const uint32_t at = from + at_s[0] + (r - row[0]) * (D / 16) + 2 * up;
        uint32_t sf;
        asm volatile("ld.shared.u16 %0, [%1];" : "=r"(sf) : "r"(at));
        if (nan_codes(sf) != 0u && ((r >= at_slot[0] && r < at_slot[1]) || (r >= at_slot[2] && r < at_slot[3]))) {
          asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"((uint16_t)without_nan(sf)) : "memory");
          odd = true;
        }
      }
      if (__any_sync(0xffffffffu, odd) && lane == 0) leave_note<T::CG>(note);
    }
    uint4 codes[kUnits];       // every step's, so that their latencies overlap
    uint32_t sfs[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(codes[i].x), "=r"(codes[i].y), "=r"(codes[i].z), "=r"(codes[i].w)
                   : "r"(from + at_c[i]));
      asm volatile("ld.shared.u16 %0, [%1];" : "=r"(sfs[i]) : "r"(from + at_s[i]));
    }
    if (use > 0 && gave_up(&freed[x], use - 1)) return false;
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const uint4 c = codes[i];
      uint32_t sf = sfs[i];
      if ((uint32_t)(row[i] - first) >= seen || !((bits >> (4 * (row[i] >> lane_sh))) & 1u)) sf = 0u;
      const uint32_t s2 = e4m3x2_to_f16x2(sf);
      const uint32_t sx[2] = {prmt(s2, 0, flip ? 0x3232 : 0x1010), prmt(s2, 0, flip ? 0x1010 : 0x3232)};
      const uint32_t w[4] = {flip ? c.z : c.x, flip ? c.w : c.y, flip ? c.x : c.z, flip ? c.y : c.w};
      const uint32_t to = at_t[i] ^ (flip ? 32u : 0u);
#pragma unroll
      for (int u = 0; u < 4; ++u)
        *reinterpret_cast<uint4*>(tile + (to ^ (16 * u))) = dequant8(w[u], sx[u >> 1]);
    }
    fence_proxy_async_smem();
    warp_arrive<T::CG>(&ready[x]);
    return true;
  }
};

// A converter's bounded wait for the inspector to come past marked chunk n: true when it gave up.
__device__ __forceinline__ bool not_inspected(const uint32_t* past, uint32_t n) {
  auto there = [&]() {
    uint32_t x;
    asm volatile("ld.acquire.cta.shared::cta.u32 %0, [%1];" : "=r"(x) : "r"(smem_u32(past)) : "memory");
    return x > n;
  };
  bool ok = there();
  if (!ok) {
    const unsigned long long t0 = now_ns();
    while (!(ok = there()) && now_ns() - t0 <= kWaitNs) {
    }
  }
  return __any_sync(0xffffffffu, !ok);
}
template <class T>
__device__ __forceinline__ bool inspect_all(const Shape& sh, const Work& p, const Span& span, uint8_t* ring,
                                            uint64_t* full, uint64_t* empty, const volatile uint32_t* copied,
                                            uint32_t* past, uint32_t* note) {
  const int lane = threadIdx.x & 31;
  constexpr int kWords = T::D / 64;                      // scales of a token
  int slot = 0, use = 0;
  uint32_t chunks = 0;
  Cursor cursor(span);
  Seg seg;
  while (cursor.next(sh, p.seqlens, seg)) {
#pragma unroll 1
    for (int c = 0; c < seg.todo; ++c, ++chunks) {
      if (gave_up(&full[slot], use)) return false;
      if (copied[slot] & kMarked) {
        const int tok0 = (seg.chunk0 + c) * T::kTok;
        uint32_t* v = reinterpret_cast<uint32_t*>(ring + slot * T::kStage + T::kKPart + T::kVCodes);
        uint32_t odd = 0u;
        // (between lo_most and n_least all see them)
#pragma unroll 1
        for (int side = 0; side < 2; ++side) {
          const int from = max((side ? seg.n_least : seg.lo_all) - tok0, 0);
          const int to = min((side ? seg.n_all : seg.lo_most) - tok0, T::kTok);
#pragma unroll 2
          for (int x = from * kWords + lane; x < to * kWords; x += 32) {
            const uint32_t w = v[x], bad = nan_codes(w);
            if (bad) v[x] = without_nan(w);
            odd |= bad;
          }
        }
        if (__any_sync(0xffffffffu, odd != 0u)) {
          if (lane == 0) *note = 1u;
          fence_proxy_async_smem();                      // (ahead of the stage's next copies)
        }
        __syncwarp();
        if (lane == 0)
          asm volatile("st.release.cta.shared::cta.u32 [%0], %1;" ::"r"(smem_u32(past)), "r"(chunks + 1u) : "memory");
      }
      __syncwarp();
      if (lane == 0) ws_arrive(&empty[slot]);
      if (++slot == T::kDepth) {
        slot = 0;
        ++use;
      }
    }
  }
  return true;
}

// ---- values that are not finite: what vectors get in the end ------------------------
// By all threads: for the CTA's vectors of each of its parts, NaN in the dims of the NaN codes (or scales) of the
// tokens that they see and others do not, where their output or their record is.  Sixteen dims of a vector a thread.
template <class T>
__device__ __forceinline__ void add_not_finite(const Shape& sh, const Work& p, int worker, int rank) {
  const Geom& g = sh.g;
  const int psh = 31 - __clz(g.P);
  const float nan = __uint_as_float(0x7FC00000u);
  Cursor cursor(plan_span<T::kThreads>(sh, p.seqlens, worker, sh.ctas));
  Seg seg;
  while (cursor.next(sh, p.seqlens, seg)) {
    const bool whole = seg.begins && seg.ends;
    float* rec = p.records + ((size_t)worker * 2 + (seg.begins ? 1 : 0)) * record_floats(sh.vt, T::D) + 2 * sh.vt;
#pragma unroll 1
    for (int x = threadIdx.x; x < T::kTiles * 128 * (T::D / 16); x += T::kThreads) {
      const int row = x / (T::D / 16), d0 = 16 * (x % (T::D / 16));
      const int at = ((row >> 7) * T::CG + rank) * 128 + (row & 127);
      if (at >= seg.vecs) continue;
      const int vec = seg.vec0 + at, j = row_of(sh, vec), head = seg.kvh * sh.G + vec - j * sh.G;
      const int n = visible_tokens(seg.L, g.R, j, g.MB * g.P), lo = first_seen(n, sh.window);
      __nv_bfloat16* out = p.out + (((size_t)seg.b * g.R + j) * g.Hq + head) * T::D;
      if (!QSA_IN_BOUNDS(seg.b < g.B && j < g.R && head < g.Hq, kChkOut) ||
          !QSA_IN_BOUNDS(worker < sh.ctas && at < sh.vt, kChkRecord))
        continue;
      const int to = min(n, (seg.chunk0 + seg.todo) * T::kTok);
#pragma unroll 1
      for (int tok = max(lo, seg.chunk0 * T::kTok); tok < to; ++tok) {
        if (tok >= seg.lo_most && tok < seg.n_least) tok = seg.n_least;       // (all see these)
        if (tok >= to) break;
        const int page = __ldg(p.page_table + (size_t)seg.b * g.MB + (tok >> psh));
        if (page < 0 || page >= g.NP) continue;
        const size_t at_tok = (((size_t)page * g.Hkv + seg.kvh) << psh) + (tok & (g.P - 1));
        const uint8_t* codes = T::E8 ? p.v_pool + at_tok * T::D + d0 : p.v_sf + at_tok * (T::D / 16) + d0 / 16;
        if constexpr (T::E8) {
          const uint4 c = *reinterpret_cast<const uint4*>(codes);
          if ((nan_codes(c.x) | nan_codes(c.y) | nan_codes(c.z) | nan_codes(c.w)) == 0u) continue;
        }
#pragma unroll 1
        for (int d = d0; d < d0 + 16; ++d) {
          if ((codes[T::E8 ? d - d0 : 0] & 0x7F) != 0x7F) continue;
          if (whole) out[d] = __float2bfloat16_rn(nan);
          else rec[((size_t)(d >> 2) * sh.vt + at) * 4 + (d & 3)] = nan;
        }
      }
    }
  }
}

// ---- 8-bit pages -----------------------------------------------------------------
// e4m3 codes with a power of two per 16 tokens (qsa_dense8.cu): codes become fp16 as they are,
// without a product, and the softmax threads have the scales: a block's power of two of K
// in the factor of its logits, that of V in the exponent of its weights, taken out
// again from the sum of the block's weights.  The copy warp brings the exponents, which are
// too short for bulk copies, as the floats that the softmax takes (bytes, taken apart by every
// thread of it, made a chunk's turn 600 cycles longer for a tile).
//
// Measured (GB300): two context chunks of 512 rows, 32 heads on 4 of 128, behind 14000 to 16384 tokens 207 us
// (1.21 PFLOP/s; NVFP4 pages 182: their codes are half the bytes to read from shared memory, and their
// scales are gone before the softmax; without the second kernel that joins the parts 190); 4 x 256 rows of
// 24 heads on 2 of 256 over 16384 306 us, 1.34 PFLOP/s; windowed verify rows (32 requests x 4 rows, 24 heads
// on 2 of 256, window 4096) 45.7 us for 138 MB, 4 to 5 of them the join.
//
// A lane has a 16-byte piece (16 codes, two 16-byte pieces of the tile) per step; a row's pieces belong to
// neighbouring lanes, of eight of them the upper four store their two in the other order
// (their 64-dim block has the same banks).  (Loads of the piece's halves in the order of their
// stores, without the selects, have conflicts of their own: 227 us for 224.)
template <class T, int kRows, int kDims>
struct Converter8 {
  static constexpr int D = T::D;
  static constexpr int kPieces = kDims / 16;                  // 16-byte pieces of a row
  static constexpr int kUnits = kRows * kPieces / 128;        // steps of a warp
  static constexpr int kStepRows = 128 / kPieces;             // rows from one step to the next
  static constexpr int kBlk = kRows * 128, kBytes = kRows * kDims * 2;
  static_assert(kStepRows % 8 == 0, "a step keeps a row's place in the swizzle");

  uint8_t* tiles;
  uint64_t *ready, *freed;
  uint32_t part, at_c, at_t;     // the stage's codes; the lane's first piece there and in the tile
  uint32_t all;                  // a chunk's copies: bit 4 i for the i-th
  int row0, lane_sh, row;

  __device__ __forceinline__ Converter8(const Shape& sh, bool v, int token0, int dim0, int dw, uint8_t* ring,
                                        uint8_t* tiles_, uint64_t* ready_, uint64_t* freed_)
      : tiles(tiles_), ready(ready_), freed(freed_), part(smem_u32(ring) + (v ? T::kKPart : 0)), row0(token0) {
    const int lane = threadIdx.x & 31, piece = lane % kPieces;
    lane_sh = 31 - __clz(min(sh.g.P, kRows));                 // log2 of a copy's rows
    row = (32 / kPieces) * dw + lane / kPieces;
    const int copies = kRows >> lane_sh;
    all = 0x1111u & ((1u << (4 * copies)) - 1u);
    const uint32_t flip = kPieces >= 8 && (lane & 4) ? 1u : 0u;
    at_c = row * D + dim0 + 16 * piece;
    at_t = ((piece >> 2) * kBlk + sw128(row, 2 * (piece & 3))) ^ (16 * flip);
  }
  __device__ __forceinline__ bool convert(const Seg& seg, int tok0, int chunks, int slot, uint32_t copied,
                                          bool v, uint32_t* note) {
    const int x = chunks & 1, use = chunks >> 1;
    uint8_t* tile = tiles + x * kBytes;
    const uint32_t from = part + slot * T::kStage + at_c;
    uint2 codes[kUnits][2];    // every step's, so that their latencies overlap; the half to be stored first
#pragma unroll
    for (int i = 0; i < kUnits; ++i)
      asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(codes[i][0].x), "=r"(codes[i][0].y), "=r"(codes[i][1].x), "=r"(codes[i][1].y)
                   : "r"(from + i * kStepRows * D));
    const bool flip = kPieces >= 8 && (threadIdx.x & 4);
    // rows that no vector of the unit sees, and what was not copied, are zeros (a code may be NaN)
    const int first = seg.lo_all - tok0 - row0, seen = max(seg.n_all - seg.lo_all, 0);
    const uint32_t bits = copied >> (v ? 2 : 0);
    if (first > 0 || first + seen < kRows || (bits & all) != all) {
#pragma unroll
      for (int i = 0; i < kUnits; ++i) {
        const int r = row + i * kStepRows;
        if ((uint32_t)(r - first) >= (uint32_t)seen || !((bits >> (4 * (r >> lane_sh))) & 1u))
          codes[i][0] = codes[i][1] = make_uint2(0u, 0u);
      }
    }
    if (use > 0 && gave_up(&freed[x], use - 1)) return false;
#pragma unroll
    for (int i = 0; i < kUnits; ++i)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint2 c = flip ? codes[i][u ^ 1] : codes[i][u];
        *reinterpret_cast<uint4*>(tile + ((at_t + i * (kStepRows / 8) * 1024) ^ (16 * u))) =
            make_uint4(e4m3x2_to_f16x2(c.x & 0xFFFFu), e4m3x2_to_f16x2(c.x >> 16), e4m3x2_to_f16x2(c.y & 0xFFFFu),
                       e4m3x2_to_f16x2(c.y >> 16));
      }
    if (v && any_partly(seg, tok0, T::kTok)) {
      bool odd = false;
#pragma unroll 1
      for (int i = 0; i < 2 * kUnits; ++i) {               // this lane's pieces as stored
        uint4* at = reinterpret_cast<uint4*>(tile + ((at_t + (i >> 1) * (kStepRows / 8) * 1024) ^ (16 * (i & 1))));
        const uint4 y = *at;
        if (partly_seen(seg, tok0 + row + (i >> 1) * kStepRows) &&
            ((not_finite2(y.x) | not_finite2(y.y) | not_finite2(y.z) | not_finite2(y.w)) & 0x80008000u)) {
          *at = make_uint4(finite2(y.x), finite2(y.y), finite2(y.z), finite2(y.w));
          odd = true;
        }
      }
      if (__any_sync(0xffffffffu, odd) && (threadIdx.x & 31) == 0) leave_note<T::CG>(note);
    }
    fence_proxy_async_smem();
    warp_arrive<T::CG>(&ready[x]);
    return true;
  }
};

// Every chunk through one converter, or through K's and then V's.
template <class T, class... C>
__device__ __forceinline__ bool convert_all(const Shape& sh, const Work& p, const Span& span, uint64_t* full,
                                            uint64_t* empty, const volatile uint32_t* copied, bool v,
                                            uint32_t* note, const uint32_t* past, C... conv) {
  int chunks = 0, slot = 0, use = 0;
  Cursor cursor(span);
  Seg seg;
  while (cursor.next(sh, p.seqlens, seg)) {
#pragma unroll 1
    for (int c = 0; c < seg.todo; ++c) {
      if (gave_up(&full[slot], use)) return false;
      const uint32_t bits = copied[slot];
      if constexpr (T::kInspect)
        if ((bits & kMarked) && not_inspected(past, chunks)) return false;
      bool second = v;
      auto one = [&](auto& cv) {
        const bool done = cv.convert(seg, (seg.chunk0 + c) * T::kTok, chunks, slot, bits, second, note);
        second = true;
        return done;
      };
      if (!(one(conv) && ...)) return false;
      // (its lanes' loads are done: warp_arrive's __syncwarp lies behind them)
      if ((threadIdx.x & 31) == 0) ws_arrive(&empty[slot]);
      if (++slot == T::kDepth) {
        slot = 0;
        ++use;
      }
      ++chunks;
    }
  }
  if ((threadIdx.x & 31) == 0) note[1] = (uint32_t)chunks;
  return true;
}

template <int D, int CG, bool E8>
__global__ void __launch_bounds__(TT<D, CG, E8>::kThreads, 1)
dense_tile_kernel(const __grid_constant__ Shape sh, const __grid_constant__ Work p) {
  using T = TT<D, CG, E8>;
  constexpr int kTok = T::kTok, kTiles = T::kTiles;
  const Geom& g = sh.g;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = CG == 2 ? (int)(blockIdx.x & 1) : 0;          // CTA of the pair
  const int worker = (int)blockIdx.x / CG;                       // whose part of the work

  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem;                                   // [kTiles][kQBytes]
  uint8_t* sK = sQ + kTiles * T::kQBytes;               // [2][kKBytes]
  uint8_t* sV = sK + 2 * T::kKBytes;                    // [2][kVBytes]
  uint8_t* ring = sV + 2 * T::kVBytes;                  // [kDepth][kStage]
  uint64_t* bars = reinterpret_cast<uint64_t*>(ring + T::kRing);
  uint64_t* kready = bars;
  uint64_t* vready = bars + 2;
  uint64_t* kfree = bars + 4;
  uint64_t* vfree = bars + 6;
  uint64_t* barS = bars + 8;
  uint64_t* pready = bars + 10;      // [buffer][half]
  uint64_t* barO = bars + 14;
  uint64_t* qready = bars + 15;
  uint64_t* mdone = bars + 16;       // after a give-up: every MMA issued has completed
  uint64_t* partO = bars + 17;
  uint64_t* full = bars + 18;        // [kDepth]
  uint64_t* empty = full + T::kDepth;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bars + T::kBars);
  uint32_t* copied = s_tmem + 4;                               // [kDepth]
  float* exps = reinterpret_cast<float*>(copied + 4);          // [kExpSlots][2^ke, ve, 2^-ve]
  // NVFP4: behind where the tokens of each marked stage lie, the chunk that the inspector has last come past, from 1 on
  [[maybe_unused]] uint32_t* past = copied + 5 * T::kDepth;

  if (tid == 0) {
    for (int x = 0; x < 2; ++x) {
      mbar_init(&kready[x], 4 * CG);
      mbar_init(&vready[x], 4 * CG);
      mbar_init(&kfree[x], 1);
      mbar_init(&vfree[x], 1);
      mbar_init(&barS[x], 1);
      mbar_init(&pready[2 * x], 4 * CG);
      mbar_init(&pready[2 * x + 1], 4 * CG);
    }
    mbar_init(barO, 1);
    mbar_init(partO, 1);
    mbar_init(mdone, 1);
    s_tmem[1] = 0u;   // set when a CTA of the pair gave up
    s_tmem[2] = 0u;   // set when V has values that are not finite
    s_tmem[3] = 0u;   // chunks of the CTA in all, when it is done
    if constexpr (!E8) *past = 0u;
    mbar_init(qready, T::kSoft * CG);
    for (int x = 0; x < T::kDepth; ++x) {
      mbar_init(&full[x], 1);
      mbar_init(&empty[x], T::kDeq + (T::kInspect ? 1 : 0));
    }
    fence_mbar_init();
  }
  if (warp == 0) {
    if constexpr (CG == 1) {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       smem_u32(s_tmem)), "r"(512u));
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    } else {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       smem_u32(s_tmem)), "r"(512u));
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
  }
  tc_fence_before();
  if constexpr (CG == 2) cluster_sync();    // the pair's barriers are initialised
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  pdl_wait();
  const Span span = plan_span<T::kThreads>(sh, p.seqlens, worker, sh.ctas);
  pdl_trigger();
  if (tid == 0 && rank == 0) describe_none(sh, p, worker);
  bool dead = false;

  if (warp < T::kSoft) {
    // ==== softmax ==================================================================
    regs_up<T::kSoftRegs>();
    const int t = warp >> 2, row = tid & 127;
    const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t tO = tmem + T::kOCol + t * D + lane_off;
    uint8_t* q_tile = sQ + t * T::kQBytes;
    const int psh = 31 - __clz(g.P);                   // log2 of the page size
    const uint32_t all_live = (1u << (kTok >> psh)) - 1u;   // (a chunk is one to four pages)
    int chunks = 0, s_waits = 0, parts = 0;   // chunks, waits on barS (two tiles), parts so far
    Cursor cursor(span);
    Seg seg;
    while (!dead && cursor.next(sh, p.seqlens, seg)) {
      // this thread's vector, its Q row as fp16 scaled by a power of two into [256, 512)
      const int at = (t * CG + rank) * 128 + row;          // its number within the unit
      const int vec = seg.vec0 + at;
      const bool real = at < seg.vecs;
      const int j = real ? row_of(sh, vec) : 0, head = seg.kvh * sh.G + (real ? vec - j * sh.G : 0);
      const size_t orow = ((size_t)seg.b * g.R + j) * g.Hq + head;
      const int n = real ? visible_tokens(seg.L, g.R, j, g.MB * g.P) : 0;
      const int lo = first_seen(n, sh.window);
      // Q rows as fp16, each scaled by a power of two into [256, 512).  The warp's 32 rows are
      // copied into the place of its own, 128 dims at a time (eight lanes to a row, all copies in
      // flight); then each thread has a row, finds its largest value and turns the row into fp16,
      // in place or, for the A operand in tensor memory, in its lane, two dims a column.  In
      // loops, not unrolled: the code runs once per part, and the instructions' own way to the
      // SM took most of its time.
      const uint32_t orow32 = (uint32_t)orow;     // (at most 2^24 rows of 256 heads)
      auto q_at = [&](int r, int pc) {            // 16-byte piece of a row of the warp
        return T::kQTmem ? q_tile + (warp & 3) * 8192 + r * 256 + ((pc ^ (r & 7)) << 4)
                         : q_tile + (pc >> 3) * 16384 + sw128(32 * (warp & 3) + r, pc & 7);
      };
      const uint32_t tQ = tmem + T::kQCol + lane_off;
      __nv_bfloat162 top2 = __float2bfloat162_rn(0.f);
      // A warp without a vector only keeps step with the barriers: its rows of S, P and O are
      // nobody's.  (With two tiles most warps have one, and the registers for asking cost more:
      // two context chunks 634 us without, 643 with it.)
      const bool some = kTiles == 2 || (t * CG + rank) * 128 + 32 * (warp & 3) < seg.vecs;
      if constexpr (!T::kPass) {
        const uint4* from = reinterpret_cast<const uint4*>(p.q + (real ? orow * D : 0));
#pragma unroll 1
        for (int d0 = 0; d0 < D && some; d0 += 128) {
          uint4 x[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = real ? from[d0 / 8 + i] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
          for (int c4 = 0; c4 < 4; ++c4) {
            uint32_t v[16];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const uint4 y = x[4 * c4 + u];
              v[4 * u] = y.x; v[4 * u + 1] = y.y; v[4 * u + 2] = y.z; v[4 * u + 3] = y.w;
            }
#pragma unroll
            for (int k = 0; k < 16; ++k)
              top2 = __hmax2(top2, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&v[k])));
            tmem_st16u(tQ + d0 / 2 + 16 * c4, v);
          }
        }
      }
#pragma unroll 1
      for (int d0 = 0; d0 < D && some && T::kPass; d0 += 128) {
        __syncwarp();
#pragma unroll 4
        for (int i = 0; i < 16; ++i) {
          const int r = 2 * i + (lane >> 4), pc = lane & 15;
          const uint32_t from = __shfl_sync(0xffffffffu, orow32, r);
          const bool there = (t * CG + rank) * 128 + 32 * (warp & 3) + r < seg.vecs;
          cp_async16(smem_u32(q_at(r, pc)), p.q + (there ? (size_t)from * D + d0 + 8 * pc : 0), there);
        }
        cp_async_wait_all();
        __syncwarp();
#pragma unroll 1
        for (int c4 = 0; c4 < 4; ++c4) {
          uint32_t v[16];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const uint4 x = *reinterpret_cast<const uint4*>(q_at(lane, 4 * c4 + u));
            v[4 * u] = x.x; v[4 * u + 1] = x.y; v[4 * u + 2] = x.z; v[4 * u + 3] = x.w;
          }
#pragma unroll
          for (int k = 0; k < 16; ++k)
            top2 = __hmax2(top2, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&v[k])));
          if constexpr (T::kQTmem) tmem_st16u(tQ + d0 / 2 + 16 * c4, v);
        }
      }
      const float amax = fmaxf(__low2float(top2), __high2float(top2));
      const int ebits = (int)((__float_as_uint(amax) >> 23) & 0xFF);
      int sq = (amax > 0.f) ? 135 - ebits : 0;
      sq = sq > 126 ? 126 : (sq < -126 ? -126 : sq);
      const float up = __uint_as_float((uint32_t)(sq + 127) << 23);
      float cq = logit_factor(p, sq);
      // (times a block's power of two it stays above zero and finite: a masked logit stays -inf)
      if constexpr (E8) cq = fminf(fmaxf(cq, 0x1p-117f), 0x1p62f);
      auto half2_of = [&](uint32_t w) {
        return pack_half2(__uint_as_float(w << 16) * up, __uint_as_float(w & 0xFFFF0000u) * up);
      };
      if constexpr (T::kQTmem) {
        tmem_wait_st();
#pragma unroll 1
        for (int c = 0; c < D / 2 && some; c += 16) {
          float raw[16];
          uint32_t v[16];
          tmem_ld16(tQ + c, raw);
          tmem_wait_ld_of(raw);
#pragma unroll
          for (int k = 0; k < 16; ++k) v[k] = half2_of(__float_as_uint(raw[k]));
          tmem_st16u(tQ + c, v);
        }
      } else {
#pragma unroll 2
        for (int pc = 0; pc < 16 && some; ++pc) {
          uint4* at_q = reinterpret_cast<uint4*>(q_at(lane, pc));
          const uint4 x = *at_q;
          *at_q = make_uint4(half2_of(x.x), half2_of(x.y), half2_of(x.z), half2_of(x.w));
        }
      }
      if constexpr (T::kQTmem) tmem_wait_st();
      else fence_proxy_async_smem();
      tc_fence_before();
      warp_arrive<CG>(qready);

      // Which pages are there: a bit per block, of 32 blocks from blk0 and of the 32 behind
      // them.  (Looked up chunk by chunk the load's latency would be on every chunk's path.)
      int blk0 = (seg.chunk0 * kTok) >> psh;
      auto there_of = [&](int beta) {
        int page = -1;
        if (beta < g.MB) page = __ldg(p.page_table + (size_t)seg.b * g.MB + beta);
        return __ballot_sync(0xffffffffu, page >= 0 && page < g.NP);
      };
      uint32_t there0 = there_of(blk0 + lane), there1 = there_of(blk0 + 32 + lane);
      float base = kNoBase;
      [[maybe_unused]] float most = -INFINITY;
      RowSum sum;
      float2 part = make_float2(0.f, 0.f);                 // the chunk's weights
      for (int c = 0; c < seg.todo; ++c, ++chunks) {
        const int y = kTiles == 2 ? t : chunks & 1;      // S buffer
        const uint32_t tS = tmem + y * kTok + lane_off;
        const int tok0 = (seg.chunk0 + c) * kTok;
        if ((tok0 >> psh) - blk0 >= 32) {
          blk0 += 32;
          there0 = there1;
          there1 = there_of(blk0 + 32 + lane);
        }
        const uint32_t live = __funnelshift_r(there0, there1, (tok0 >> psh) - blk0);   // the chunk's blocks
        if (gave_up(&barS[y], kTiles == 2 ? s_waits : chunks >> 1)) { dead = true; break; }
        ++s_waits;
        tc_fence_after();
        if (!some) {
          tc_fence_before();
#pragma unroll
          for (int h = 0; h < T::kHalves; ++h) warp_arrive<CG>(&pready[2 * y + h]);
          continue;
        }
        const bool edge = tok0 + kTok > seg.n_least || tok0 < seg.lo_most ||
                          (live & all_live) != all_live;
        // The blocks' scales.  (With two tiles, whose turns the softmax bounds, before the logits:
        // 220 us for 224 in 2 x 512 context rows; with one 36.4 for 35.5, 160 vectors.)
        [[maybe_unused]] float4 ex[E8 ? 6 : 1];
        auto scales = [&]() {
          const float4* from = reinterpret_cast<const float4*>(exps + T::kExpFloats * (chunks & (T::kExpSlots - 1)));
#pragma unroll
          for (int i = 0; i < 6; ++i) ex[i] = from[i];
        };
        if constexpr (E8 && kTiles == 2) scales();
        // The row's logits, those it does not see at -inf.
        float z[kTok];
#pragma unroll
        for (int i = 0; i < kTok / 32; ++i) tmem_ld32(tS + 32 * i, z + 32 * i);
        // (the chunk before's, while the loads are on their way: two context chunks 630 us; behind the weights 636)
        sum.add(part);
        tmem_wait_ld_of(z);
        if (edge) {
#pragma unroll
          for (int i = 0; i < kTok; ++i) {
            const int tok = tok0 + i;
            if (tok >= n || tok < lo || !((live >> ((i & ~31) >> psh)) & 1u)) z[i] = -INFINITY;
          }
        }
        float top;
        // A block's factor of its logits, its exponent of V (log2) and 2^-that.
        [[maybe_unused]] float bc[kTok / 16];
        auto of = [](const float4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; };
        if constexpr (E8) {
          if constexpr (kTiles == 1) scales();
          top = -INFINITY;
#pragma unroll
          for (int i = 0; i < kTok / 16; ++i) {
            bc[i] = cq * of(ex[i >> 2], i & 3);
            float m = fmaxf(z[16 * i], z[16 * i + 1]), m2 = fmaxf(z[16 * i + 2], z[16 * i + 3]);
#pragma unroll
            for (int k = 4; k < 16; k += 4) {
              m = fmax3(m, z[16 * i + k], z[16 * i + k + 1]);
              m2 = fmax3(m2, z[16 * i + k + 2], z[16 * i + k + 3]);
            }
            top = fmaxf(top, fmaf(fmaxf(m, m2), bc[i], of(ex[2 + (i >> 2)], i & 3)));
          }
        } else {
          float m8[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) m8[i] = z[i];
#pragma unroll
          for (int i = 8; i < kTok; i += 2) m8[(i >> 1) & 7] = fmax3(m8[(i >> 1) & 7], z[i], z[i + 1]);
          top = cq * fmax3(fmax3(m8[0], m8[1], m8[2]), fmax3(m8[3], m8[4], m8[5]),
                                       fmaxf(m8[6], m8[7]));
        }
        // The base moves where a logit would overflow an fp16 weight, and with it what has
        // been summed on the old one.
        // (8-bit: then for every vector of the warp, to below its largest so far, as it is the warp
        // that waits: 2 x 512 context rows with logits up to a deviation of 2 220 us before, 205
        // now, 199 where nothing moves; 4 x 256 rows of 24 heads on 2 of 256 350 and 316.  By a
        // power of two, so that what a vector has summed so far is rescaled exactly; its later weights
        // are rounded at another base, so that its last bits may hang on when its neighbours' bases move.)
        if constexpr (E8) most = fmaxf(most, top);
        bool moves = top > base + kHeadroom;
        if (__any_sync(0xffffffffu, moves)) {
          if constexpr (E8) moves = most > base + kBelow;
          const float nb = moves ? (E8 ? floorf(most) : top) - kBelow : base;
          const float alpha = exp2_approx(base - nb);
          base = nb;
          sum.scale(alpha);
          if (c > 0) {
            // with two tiles barS has said that O is complete up to the chunk before
            if (kTiles == 1 && gave_up(barO, chunks - 1)) { dead = true; break; }
            tc_fence_after();
#pragma unroll 1
            for (int i = 0; i < D / 16; ++i) {   // (rare: kept small, as the instruction cache is)
              float o16[16];
              tmem_ld16(tO + 16 * i, o16);
              tmem_wait_ld_of(o16);
#pragma unroll
              for (int u = 0; u < 16; ++u) o16[u] *= alpha;
              tmem_st16(tO + 16 * i, o16);
            }
          }
        }
        // P, 64 tokens at a time, over the first columns they were read from.
        part = make_float2(0.f, 0.f);
#pragma unroll
        for (int h = 0; h < T::kHalves; ++h) {
          float2 c2 = make_float2(cq, cq), b2 = make_float2(-base, -base);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t pk[16];
            if constexpr (E8) {
#pragma unroll
              for (int u = 0; u < 2; ++u) {       // a block of 16 tokens
                const int n16 = 4 * h + 2 * q + u;
                const float vb = of(ex[2 + (n16 >> 2)], n16 & 3) - base, back = of(ex[4 + (n16 >> 2)], n16 & 3);
                c2 = make_float2(bc[n16], bc[n16]);
                b2 = make_float2(vb, vb);
                float2 block = make_float2(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  const int k = 64 * h + 32 * q + 16 * u + 2 * i;
                  const float2 a = fma2(make_float2(z[k], z[k + 1]), c2, b2);
                  const float2 e = make_float2(exp2_approx(a.x), exp2_approx(a.y));
                  block = add2(block, e);
                  pk[8 * u + i] = pack_weights(e.x, e.y);
                }
                part = fma2(block, make_float2(back, back), part);
              }
            } else {
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const int k = 64 * h + 32 * q + 2 * i;
                const float2 a = fma2(make_float2(z[k], z[k + 1]), c2, b2);
                const float2 e = make_float2(exp2_approx(a.x), exp2_approx(a.y));
                part = add2(part, e);
                pk[i] = pack_weights(e.x, e.y);
              }
            }
            tmem_st16u(tS + 64 * h + 16 * q, pk);
          }
          tmem_wait_st();
          tc_fence_before();
          warp_arrive<CG>(&pready[2 * y + h]);
        }
      }
      if (dead) break;
      // ---- the part's output ---------------------------------------------------------
      const bool late = kTiles == 2 ? gave_up(&barS[t], s_waits) : gave_up(partO, parts);
      ++parts;
      ++s_waits;
      if (late) { dead = true; break; }
      tc_fence_after();
      sum.add(part);
      float l = sum.total(), m = base, f = 1.f;
      const bool whole = seg.begins && seg.ends;
      if (whole && p.sinks && real) {
        const float s2 = p.sinks[head] * kLog2e, nm = fmaxf(m, s2);
        f = exp2_approx(m - nm);
        l = l * f + exp2_approx(s2 - nm);
        m = nm;
      }
      const float r = whole ? (l == 0.f ? 0.f : f * p.v_scale / l) : 1.f;
      float* rec = p.records + ((size_t)worker * 2 + (seg.begins ? 1 : 0)) * record_floats(sh.vt, D);
      const bool rec_ok = QSA_IN_BOUNDS(worker < sh.ctas && at < sh.vt, kChkRecord);
      const int at0 = (t * CG + rank) * 128 + 32 * (warp & 3);    // the warp's first vector
      const int left = min(32, seg.vecs - at0);                   // and how many it has
      if (!whole) {
        // a record: four dims of neighbouring vectors behind one another, as the lanes have them
        float4* to = reinterpret_cast<float4*>(rec + 2 * sh.vt) + at;
#pragma unroll 1
        for (int d0 = 0; d0 < D && left > 0; d0 += 32) {
          float o32[32];
          tmem_ld32(tO + d0, o32);
          tmem_wait_ld_of(o32);
          if (real && rec_ok)
#pragma unroll
            for (int i = 0; i < 8; ++i)
              to[(size_t)(d0 / 4 + i) * sh.vt] =
                  make_float4(o32[4 * i], o32[4 * i + 1], o32[4 * i + 2], o32[4 * i + 3]);
        }
      } else if constexpr (!T::kPass) {
        uint32_t row4[4], rows4 = 0u;                    // the rows of this lane and its three neighbours
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          row4[k] = __shfl_sync(0xffffffffu, orow32, (lane & 28) + k);
          rows4 |= (uint32_t)((lane & 28) + k < left && QSA_IN_BOUNDS(row4[k] < (size_t)g.B * g.R * g.Hq, kChkOut))
                   << k;
        }
#pragma unroll 1
        for (int d0 = 0; d0 < D && left > 0; d0 += 32) {
          float o32[32];
          tmem_ld32(tO + d0, o32);
          tmem_wait_ld_of(o32);
          uint32_t w[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const __nv_bfloat162 y = __floats2bfloat162_rn(o32[2 * k] * r, o32[2 * k + 1] * r);
            w[k] = *reinterpret_cast<const uint32_t*>(&y);
          }
          transpose4(w, lane);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (rows4 >> k & 1u)
              *reinterpret_cast<uint4*>(p.out + (size_t)row4[k] * D + d0 + 8 * (lane & 3)) =
                  make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
        }
      } else {
        // O leaves 64 columns at a time by way of shared memory of the warp's own (its Q rows,
        // whose last reader is done), so that rows are written in runs of 128 bytes.
        // 32 rows of 64 floats, in the warp's 8 KB or in the 4 KB that its rows have of the first
        // two blocks (no other warp's: it may be writing its next Q)
        auto box = [&](int rr) {
          return T::kQTmem ? q_tile + (warp & 3) * 8192 + rr * 256
                           : q_tile + (rr >> 4) * 16384 + (warp & 3) * 4096 + (rr & 15) * 256;
        };
        const int sub = lane >> 4, pc = lane & 15;
#pragma unroll 1
        for (int d0 = 0; d0 < D && left > 0; d0 += 64) {
          float o64[64];
          tmem_ld32(tO + d0, o64);
          tmem_ld32(tO + d0 + 32, o64 + 32);
          tmem_wait_ld_of(o64);
#pragma unroll
          for (int i = 0; i < 16; ++i)       // 16-byte pieces, swizzled by the row
            *reinterpret_cast<float4*>(box(lane) + ((i ^ (lane & 15)) << 4)) =
                make_float4(o64[4 * i] * r, o64[4 * i + 1] * r, o64[4 * i + 2] * r, o64[4 * i + 3] * r);
          __syncwarp();
#pragma unroll 8
          for (int i = 0; i < 16; ++i) {   // two rows at a time, a piece per lane
            const int rr = 2 * i + sub;
            const float4 x = *reinterpret_cast<const float4*>(box(rr) + ((pc ^ (rr & 15)) << 4));
            const uint32_t to = __shfl_sync(0xffffffffu, orow32, rr);
            const __nv_bfloat162 lo2 = __floats2bfloat162_rn(x.x, x.y), hi2 = __floats2bfloat162_rn(x.z, x.w);
            if (rr < left && QSA_IN_BOUNDS(to < (size_t)g.B * g.R * g.Hq, kChkOut))
              *reinterpret_cast<uint2*>(p.out + (size_t)to * D + d0 + 4 * pc) =
                  make_uint2(*reinterpret_cast<const uint32_t*>(&lo2), *reinterpret_cast<const uint32_t*>(&hi2));
          }
          __syncwarp();
        }
      }
      if (real) {
        if (whole) {
          if (QSA_IN_BOUNDS(orow < (size_t)g.B * g.R * g.Hq, kChkOut))
            p.lse[orow] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
        } else if (rec_ok) {
          rec[at] = m;
          rec[sh.vt + at] = l;
        }
      }
      if (tid == 0 && rank == 0 && seg.ends) describe(sh, p, span, cursor, seg, worker);
    }
  } else if (warp < T::kMma) {
    // ==== dequantisation =============================================================
    regs_down<T::kDeqRegs>();
    const int dw = (warp - T::kSoft) & 3;
    using CK = std::conditional_t<E8, Converter8<T, T::kKRows, D>, Converter<T, T::kKRows, D>>;
    using CV = std::conditional_t<E8, Converter8<T, kTok, T::kVDims>, Converter<T, kTok, T::kVDims>>;
    const bool v = warp - T::kSoft >= 4;
    const int k0 = rank * T::kKRows, v0 = rank * T::kVDims;
    if constexpr (T::kDeq == 4)
      dead = !convert_all<T>(sh, p, span, full, empty, copied, false, s_tmem + 2, past,
                             CK(sh, false, k0, 0, dw, ring, sK, kready, kfree),
                             CV(sh, true, 0, v0, dw, ring, sV, vready, vfree));
    else if constexpr (CG == 1)   // one shape: one copy of the code for both
      dead = !convert_all<T>(sh, p, span, full, empty, copied, v, s_tmem + 2, past,
                             CK(sh, v, 0, 0, dw, ring, v ? sV : sK, v ? vready : kready, v ? vfree : kfree));
    else if (!v)
      dead = !convert_all<T>(sh, p, span, full, empty, copied, false, s_tmem + 2, past,
                             CK(sh, false, k0, 0, dw, ring, sK, kready, kfree));
    else
      dead = !convert_all<T>(sh, p, span, full, empty, copied, true, s_tmem + 2, past,
                             CV(sh, true, 0, v0, dw, ring, sV, vready, vfree));
  } else if (regs_down<T::kMmaRegs>(), warp == T::kMma + 1) {
    // ==== copies =====================================================================
    dead = !copy_all<T>(sh, p, span, rank, ring, full, empty, copied, exps, reinterpret_cast<int*>(copied + T::kDepth));
  } else if (T::kInspect && warp == T::kMma + 2) {
    // ==== inspection =================================================================
    if constexpr (T::kInspect) dead = !inspect_all<T>(sh, p, span, ring, full, empty, copied, past, s_tmem + 2);
  } else if (warp == T::kMma && rank == 0) {
    // ==== MMA issue ==================================================================
    const uint32_t one = elect_one();
    const uint32_t id_s = f16_idesc(128 * CG, kTok), id_o = f16_idesc(128 * CG, D) | kIdescBMn;
    Cursor cursor(span);
    Seg seg;
    int s_done = 0, parts = 0;     // chunks whose S was issued in earlier parts; parts
    auto issue_s = [&](int t, int y, int x) {
      const uint64_t dq = sw128_desc(smem_u32(sQ + t * T::kQBytes));
      const uint64_t dk = sw128_desc(smem_u32(sK + x * T::kKBytes));
#pragma unroll
      for (int h = 0; h < D / 64; ++h)
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          if constexpr (T::kQTmem)     // 16 dims (one step): 8 columns
            mma_ts<CG>(one, tmem + y * kTok, tmem + T::kQCol + 8 * (4 * h + ks),
                       dk + (uint64_t)((h * T::kKBlk + 32 * ks) >> 4), id_s, (h | ks) ? 1u : 0u);
          else
            mma_ss<CG>(one, tmem + y * kTok, dq + (uint64_t)((h * 16384 + 32 * ks) >> 4),
                       dk + (uint64_t)((h * T::kKBlk + 32 * ks) >> 4), id_s, (h | ks) ? 1u : 0u);
    };
    auto issue_o = [&](int t, int y, int x, int h, bool first) {   // 64 tokens
      const uint64_t dv = sw128_mn_desc(smem_u32(sV + x * T::kVBytes), T::kVBlk);
#pragma unroll
      for (int ks = 0; ks < 4; ++ks)
        mma_ts<CG>(one, tmem + T::kOCol + t * D, tmem + y * kTok + 64 * h + 8 * ks,
                   dv + (uint64_t)((8192 * h + 2048 * ks) >> 4), id_o,
                   (first && ks == 0) ? 0u : 1u);
    };
    while (!dead && cursor.next(sh, p.seqlens, seg)) {
      if (gave_up(qready, parts)) { dead = true; break; }
      ++parts;
      tc_fence_after();
      const int C = seg.todo;
      auto chunk_s = [&](int c) {   // waits for K of chunk c
        const int n = s_done + c, x = n & 1;
        if (gave_up(&kready[x], n >> 1)) return false;
        tc_fence_after();
        return true;
      };
      if constexpr (kTiles == 2) {
        if (!chunk_s(0)) { dead = true; break; }
        issue_s(0, 0, s_done & 1);
        commit<CG>(one, &barS[0]);
        issue_s(1, 1, s_done & 1);
        commit<CG>(one, &barS[1]);
        commit<CG>(one, &kfree[s_done & 1]);
        // The tiles of a chunk are waited for while the products before it run.
        if (gave_up(&vready[s_done & 1], s_done >> 1) || (C > 1 && !chunk_s(1))) { dead = true; break; }
        for (int c = 0; c < C && !dead; ++c) {
          const int n = s_done + c, x = n & 1, xn = (n + 1) & 1;
          const bool more = c + 1 < C;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (gave_up(&pready[2 * t], n)) { dead = true; break; }
            tc_fence_after();
            issue_o(t, t, x, 0, c == 0);
            if (gave_up(&pready[2 * t + 1], n)) { dead = true; break; }
            tc_fence_after();
            issue_o(t, t, x, 1, false);
            if (more) issue_s(t, t, xn);
            commit<CG>(one, &barS[t]);
          }
          if (dead) break;
          commit<CG>(one, &vfree[x]);
          if (more) {
            commit<CG>(one, &kfree[xn]);
            if (gave_up(&vready[xn], (n + 1) >> 1) || (c + 2 < C && !chunk_s(c + 2))) {
              dead = true;
              break;
            }
          }
        }
      } else {
        for (int c = 0; c < 2 && c < C; ++c) {
          const int n = s_done + c;
          if (!chunk_s(c)) { dead = true; break; }
          issue_s(0, n & 1, n & 1);
          commit<CG>(one, &barS[n & 1]);
          commit<CG>(one, &kfree[n & 1]);
        }
        for (int c = 0; c < C && !dead; ++c) {
          const int n = s_done + c, x = n & 1;
          if (gave_up(&vready[x], n >> 1)) { dead = true; break; }
#pragma unroll
          for (int h = 0; h < T::kHalves && !dead; ++h) {
            if (gave_up(&pready[2 * x + h], n >> 1)) { dead = true; break; }
            tc_fence_after();
            issue_o(0, x, x, h, c == 0 && h == 0);
          }
          if (dead) break;
          commit<CG>(one, &vfree[x]);
          commit<CG>(one, barO);
          if (c + 1 == C) commit<CG>(one, partO);
          if (c + 2 < C) {
            if (!chunk_s(c + 2)) { dead = true; break; }
            issue_s(0, x, x);
            commit<CG>(one, &barS[x]);
            commit<CG>(one, &kfree[x]);
          }
        }
      }
      s_done += C;
    }
  }

  // Every MMA has completed where nothing gave up (the softmax waited for the last); after a
  // give-up, wait for what the MMA warp issued before its memory goes.
  if (dead) atomicExch(p.status, kStatusWaitTimeout);
  tc_fence_before();
  bool any_dead = __syncthreads_or(dead);
  if constexpr (CG == 2) {
    // both CTAs of the pair learn of a give-up in one (the word of a barrier not used again)
    if (any_dead && tid == 0)
      asm volatile(
          "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, 0;\n\tst.shared::cluster.u32 [a], %1;\n\t"
          "mapa.shared::cluster.u32 a, %0, 1;\n\tst.shared::cluster.u32 [a], %1;\n\t}" ::"r"(
              smem_u32(s_tmem + 1)), "r"(1u)
          : "memory");
    cluster_sync();
    any_dead = s_tmem[1] != 0u;
  }
  tc_fence_after();
  if (any_dead) {
    if (warp == T::kMma && rank == 0) commit<CG>(elect_one(), mdone);
    gave_up(mdone, 0);
    __syncthreads();
  }
  if (!any_dead && warp == 0) {
    // Nor may an arrival of the MMAs' commits that nobody else waits for be on its way when the block ends: the
    // softmax warps wait for a part's last products, not for the barriers that are told of them next.  A lane
    // waits for each.
    const int chunks = (int)*reinterpret_cast<volatile uint32_t*>(s_tmem + 3), x = lane & 1;
    const bool o = lane == 4;
    uint64_t* bar = o ? barO : lane & 2 ? &vfree[x] : &kfree[x];
    if (lanes_gave_up(bar, o ? chunks - 1 : (chunks - 1 - x) >> 1, o ? kTiles == 1 && chunks > 0 : lane < 4 && x < chunks))
      atomicExch(p.status, kStatusWaitTimeout);
  }
  if (!any_dead && *reinterpret_cast<volatile uint32_t*>(s_tmem + 2) != 0u) add_not_finite<T>(sh, p, worker, rank);
  if constexpr (CG == 2) cluster_sync();
  if (warp == 0) {
    if constexpr (CG == 1)
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
    else
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
  }
}

}  // namespace
}  // namespace dense

// Pairs of CTAs where single ones would take more units: a pair's unit is 512 vectors at
// head_dim 128 and 256 at 256 (4 requests of 8192 tokens, pairs against singles: 160 vectors
// 38 and 31 us at head_dim 128, 28.9 and 29.5 at 256; 512 vectors 42 and 49, 42 and 44).
static bool use_pairs(const Geom& g) {
  return g.R * (g.Hq / g.Hkv) > (g.D == 128 ? 256 : 128);
}

dense::Shape dense_tile_shape(const Geom& g, int window) {
  dense::Shape s;
  auto set = [&](auto t) {
    using T = decltype(t);
    s.vt = T::kVecs;
    s.tok_sh = T::kTok == 128 ? 7 : 6;
    s.ctas = sm_count() / T::CG;
  };
  dense::set_heads(&s, g);
  if (use_pairs(g)) {
    if (g.D == 128) set(dense::TT<128, 2, false>());   // (8-bit pages alike)
    else set(dense::TT<256, 2, false>());
  } else {
    if (g.D == 128) set(dense::TT<128, 1, false>());
    else set(dense::TT<256, 1, false>());
  }
  s.tiles = (g.R * s.G + s.vt - 1) / s.vt;
  s.window = window;
  // A short context is divided down to two chunks (64 rows over 2048 tokens: 19.2, 21.3,
  // 24.9 us with two, four, eight); a part's start and end take what ten chunks take
  // (windowed verify rows 45.3, 43.3, 43.5, 45.0 us with 4, 7, 10, 14, 77 context rows 32.7,
  // 30.4, 29.3, 29.5).
  s.least = 2;
  s.lead = 10;
  s.by_unit = dense::unit_count(s) <= s.ctas;
  return s;
}

namespace {

template <int D, int CG, bool E8>
cudaError_t launch_tile(const dense::Shape& s, const dense::Work& w, cudaStream_t stream) {
  using T = dense::TT<D, CG, E8>;
  auto* kern = dense::dense_tile_kernel<D, CG, E8>;
  static_assert(T::kSmem + 1024 <= 227 * 1024, "shared memory (and plan_span's, which takes up 1024 bytes here)");
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, T::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(s.ctas * CG);
  cfg.blockDim = dim3(T::kThreads);
  cfg.dynamicSmemBytes = T::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CG;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CG == 2 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, s, w);
}

template <bool E8>
cudaError_t launch_tiles(const dense::Shape& s, const dense::Work& w, cudaStream_t stream) {
  if (use_pairs(s.g))
    return s.g.D == 256 ? launch_tile<256, 2, E8>(s, w, stream) : launch_tile<128, 2, E8>(s, w, stream);
  return s.g.D == 256 ? launch_tile<256, 1, E8>(s, w, stream) : launch_tile<128, 1, E8>(s, w, stream);
}

}  // namespace

cudaError_t launch_dense_tile(const dense::Shape& s, const dense::Work& w, bool e8, cudaStream_t stream) {
  return e8 ? launch_tiles<true>(s, w, stream) : launch_tiles<false>(s, w, stream);
}

}  // namespace qsa

QSA_BOUNDS_READER(bounds_word_dense_tile)
