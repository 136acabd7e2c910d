// qsa_dense_tile.cu -- dense attention over the NVFP4 paged cache for many
// query vectors per KV head (context row groups, wide verify rows), on the
// fifth-generation tensor cores.
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
// Measured (GB300, SM clock 2070 MHz):
//   two context chunks of 1024 rows, 32 heads on 4, behind 30000 tokens: 638 to 650 us,
//   1.6 PFLOP/s (0.81 of the measured cuBLAS rate).  The tensor pipe is active
//   70 % of the time: a chunk's turn takes 2940 cycles of which its MMAs need 2048,
//   the rest is the softmax's latency between a tile's turns.
//   The same at 24 heads on 2 of 256: 964 us, 1.68 PFLOP/s (0.85); 4 x 256 rows of
//   these over 16384 tokens 270 us (floor 208).
//   32 requests x 4 verify rows, 24 heads on 2, head_dim 256, window 4096: 44 us
//   for 79 MB (floor 11.8).  A CTA has 30 chunks of 64 tokens, 1780 cycles each (the K
//   warps' conversion, shared memory; the MMAs need 1024, 80 of the tile's 128 rows hold
//   no vector), a start of 5.6 us (work division 0.7,
//   queries 4.3, first pages and S 0.6), a record (1.2 us), and the join kernel with its
//   launch (9 us).  16 requests x 4 rows of 32 heads on 4 of 128 over 16384 tokens: 77 us
//   for 151 MB (floor 22.6).
//
// Roles in a CTA (a warp group each unless noted):
//   softmax   a thread per vector (tensor-memory lane): its row of S to registers, base
//             (moved only where a weight would overflow), P = exp2(S c - base) as
//             fp16 over the columns of S it has read, 64 tokens at a time, sums in fp32;
//             at the end of a part O from tensor memory to the output or to a record.  A
//             group per tile
//   copy      one warp: codes and scales of the pages by bulk copies some chunks ahead
//   dequant   e2m1 x e4m3 exact in fp16 into double-buffered K and V tiles (128-byte swizzle)
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
//   empty[i]      stage i read                                     (the converting warps)
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
#include "qsa_tc.cuh"

namespace qsa {
namespace dense {
namespace {

using namespace tc;

// Bounds-check codes (reported by bounds-checked builds only).
[[maybe_unused]] constexpr int kChkChunk = 0xA01;   // copy: token offset or place in the ring out of range
[[maybe_unused]] constexpr int kChkOut = 0xA02;     // output row out of range
[[maybe_unused]] constexpr int kChkRecord = 0xA03;  // record's slot out of range

template <int D_, int CG_>
struct TT {
  static constexpr int D = D_, CG = CG_;                 // CG: CTAs per MMA
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
  static constexpr int kQBytes = kQTmem ? 32768 : 128 * D * 2;
  // Codes and scales on their way: a stage is a chunk, this CTA's K rows and whole V rows.
  static constexpr int kDepth = CG == 2 ? 4 : 3;
  static constexpr int kKCodes = kKRows * D / 2, kVCodes = kTok * D / 2;
  static constexpr int kKPart = kKCodes + kKCodes / 8, kVPart = kVCodes + kVCodes / 8;
  static constexpr int kStage = kKPart + kVPart;
  static constexpr int kRing = kDepth * kStage;
  static constexpr int kBars = 18 + 2 * kDepth;
  static constexpr int kSmem = 1024 + kTiles * kQBytes + 2 * kKBytes + 2 * kVBytes + kRing +
                               kBars * 8 + 16 + kDepth * 4;
};

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

// Asynchronous copy of 16 bytes, zeros where `on` is false.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

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
                                         volatile uint32_t* copied) {
  const int lane = threadIdx.x & 31;
  const int psh = 31 - __clz(sh.g.P);
  const bool scales = lane & 1, v = lane & 2;
  const int rows = v ? T::kTok : T::kKRows;
  const int step = min(sh.g.P, rows);                 // rows of a copy
  const int off = (lane >> 2) * step;                 // its first, in the stage's part
  const bool mine = lane < 8 && off < rows;
  const int tok_off = off + (v ? 0 : rank * T::kKRows);
  const uint32_t row_bytes = scales ? T::D / 16 : T::D / 2, bytes = step * row_bytes;
  const uint8_t* pool = v ? (scales ? p.v_sf : p.v_pool) : (scales ? p.k_sf : p.k_pool);
  uint8_t* dst = ring + (v ? T::kKPart + (scales ? T::kVCodes : 0) : (scales ? T::kKCodes : 0)) +
                 off * row_bytes;
  const uint64_t policy = policy_evict_normal();   // (other units read the page too)
  int slot = 0, use = 0;
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
      if (lane == 0) {
        copied[slot] = which;
        mbar_arrive_expect_tx(&full[slot], sum);
      }
      __syncwarp();
      if (there)
        bulk_g2s(dst + slot * T::kStage,
                 pool + ((((size_t)page * sh.g.Hkv + seg.kvh) << psh) + (tok & (sh.g.P - 1))) * row_bytes,
                 bytes, &full[slot], policy);
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
                                          bool v) {
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

// Every chunk through one converter, or through K's and then V's.
template <class T, class... C>
__device__ __forceinline__ bool convert_all(const Shape& sh, const Work& p, const Span& span, uint64_t* full,
                                            uint64_t* empty, const volatile uint32_t* copied, bool v,
                                            C... conv) {
  int chunks = 0, slot = 0, use = 0;
  Cursor cursor(span);
  Seg seg;
  while (cursor.next(sh, p.seqlens, seg)) {
#pragma unroll 1
    for (int c = 0; c < seg.todo; ++c) {
      if (gave_up(&full[slot], use)) return false;
      const uint32_t bits = copied[slot];
      bool second = v;
      auto one = [&](auto& cv) {
        const bool done = cv.convert(seg, (seg.chunk0 + c) * T::kTok, chunks, slot, bits, second);
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
  return true;
}

template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

template <int D, int CG>
__global__ void __launch_bounds__(TT<D, CG>::kThreads, 1)
dense_tile_kernel(const __grid_constant__ Shape sh, const __grid_constant__ Work p) {
  using T = TT<D, CG>;
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
    mbar_init(qready, T::kSoft * CG);
    for (int x = 0; x < T::kDepth; ++x) {
      mbar_init(&full[x], 1);
      mbar_init(&empty[x], T::kDeq);
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
#pragma unroll 1
      for (int d0 = 0; d0 < D && some; d0 += 128) {
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
      const float cq = logit_factor(p, sq);
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
      float2 sum = make_float2(0.f, 0.f);
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
        // The row's logits, those it does not see at -inf.
        float z[kTok];
#pragma unroll
        for (int i = 0; i < kTok / 32; ++i) tmem_ld32(tS + 32 * i, z + 32 * i);
        tmem_wait_ld_of(z);
        if (edge) {
#pragma unroll
          for (int i = 0; i < kTok; ++i) {
            const int tok = tok0 + i;
            if (tok >= n || tok < lo || !((live >> ((i & ~31) >> psh)) & 1u)) z[i] = -INFINITY;
          }
        }
        float m8[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) m8[i] = z[i];
#pragma unroll
        for (int i = 8; i < kTok; i += 2) m8[(i >> 1) & 7] = fmax3(m8[(i >> 1) & 7], z[i], z[i + 1]);
        const float top = cq * fmax3(fmax3(m8[0], m8[1], m8[2]), fmax3(m8[3], m8[4], m8[5]),
                                     fmaxf(m8[6], m8[7]));
        // The base moves where a logit would overflow an fp16 weight, and with it what has
        // been summed on the old one.
        const bool moves = top > base + kHeadroom;
        if (__any_sync(0xffffffffu, moves)) {
          const float nb = moves ? top - kBelow : base;
          const float alpha = exp2_approx(base - nb);
          base = nb;
          sum.x *= alpha;
          sum.y *= alpha;
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
#pragma unroll
        for (int h = 0; h < T::kHalves; ++h) {
          const float2 c2 = make_float2(cq, cq), b2 = make_float2(-base, -base);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int k = 64 * h + 32 * q + 2 * i;
              const float2 a = fma2(make_float2(z[k], z[k + 1]), c2, b2);
              const float2 e = make_float2(exp2_approx(a.x), exp2_approx(a.y));
              sum = add2(sum, e);
              pk[i] = pack_weights(e.x, e.y);
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
      float l = sum.x + sum.y, m = base, f = 1.f;
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
    using CK = Converter<T, T::kKRows, D>;
    using CV = Converter<T, kTok, T::kVDims>;
    const bool v = warp - T::kSoft >= 4;
    const int k0 = rank * T::kKRows, v0 = rank * T::kVDims;
    if constexpr (T::kDeq == 4)
      dead = !convert_all<T>(sh, p, span, full, empty, copied, false,
                             CK(sh, false, k0, 0, dw, ring, sK, kready, kfree),
                             CV(sh, true, 0, v0, dw, ring, sV, vready, vfree));
    else if constexpr (CG == 1)   // one shape: one copy of the code for both
      dead = !convert_all<T>(sh, p, span, full, empty, copied, v,
                             CK(sh, v, 0, 0, dw, ring, v ? sV : sK, v ? vready : kready, v ? vfree : kfree));
    else if (!v)
      dead = !convert_all<T>(sh, p, span, full, empty, copied, false,
                             CK(sh, false, k0, 0, dw, ring, sK, kready, kfree));
    else
      dead = !convert_all<T>(sh, p, span, full, empty, copied, true,
                             CV(sh, true, 0, v0, dw, ring, sV, vready, vfree));
  } else if (regs_down<T::kMmaRegs>(), warp == T::kMma + 1) {
    // ==== copies =====================================================================
    dead = !copy_all<T>(sh, p, span, rank, ring, full, empty, copied);
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
static bool use_pairs(const Geom& g) { return g.R * (g.Hq / g.Hkv) > (g.D == 128 ? 256 : 128); }

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
    if (g.D == 128) set(dense::TT<128, 2>());
    else set(dense::TT<256, 2>());
  } else {
    if (g.D == 128) set(dense::TT<128, 1>());
    else set(dense::TT<256, 1>());
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

template <int D, int CG>
cudaError_t launch_tile(const dense::Shape& s, const dense::Work& w, cudaStream_t stream) {
  using T = dense::TT<D, CG>;
  auto* kern = dense::dense_tile_kernel<D, CG>;
  static_assert(T::kSmem <= 227 * 1024, "shared memory");
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

}  // namespace

cudaError_t launch_dense_tile(const dense::Shape& s, const dense::Work& w, cudaStream_t stream) {
  if (use_pairs(s.g))
    return s.g.D == 256 ? launch_tile<256, 2>(s, w, stream) : launch_tile<128, 2>(s, w, stream);
  return s.g.D == 256 ? launch_tile<256, 1>(s, w, stream) : launch_tile<128, 1>(s, w, stream);
}

}  // namespace qsa

QSA_BOUNDS_READER(bounds_word_dense_tile)
