// qsa_prompt.cu -- attention over whole prompts, packed behind one another, before
// (or without) a cache: bf16 queries, keys and values, causal, grouped heads, windows and
// sinks, on the fifth-generation tensor cores.
//
//   z_t = sm_scale q.K_t,  out = sum_{t <= row} exp(z_t - lse) V_t
//
// 4 D flops per (query vector, token that it sees) on the tensor core bound it; keys and
// values of one KV head pass through L2.
//   S = Q K^T    A = Q, B = K from shared memory (K-major), S in tensor memory
//   O += P V     A = P from tensor memory, B = V from shared memory (token rows, MN-major)
// A tile is 128 query vectors of one sequence and KV head: floor(128 / G) rows times the G
// heads that share it, as one TMA box brings them, so that a chunk of keys is read once for
// all its heads and short sequences still fill tiles.  A unit is the tiles of a pair of CTAs
// (cta_group::2: each SM has half of every K and V tile, and feeds half of the B operand): four
// at head_dim 128, two at 256.  It walks its chunks of 128 tokens from the first that its rows see up to
// the last row's own.
//
// Units of one sequence differ in length (causal).  They are dealt to the pairs longest first,
// there and back: the r-th turn goes to pairs 0, 1, ... where r is even and ..., 1, 0 where it
// is odd, so that all end within about a unit's difference, without a ticket or a message; the copy warp of
// each CTA finds them and leaves them to the other roles.
//
// Weights are bf16, as V is (one kind of operand per MMA): eight bits each, of sums that are fp32.
// bf16 has fp32's exponents, so no weight is lost to the base; it is the exact maximum of the first
// tokens, and moves when a later logit is 2^8 above it.  (Two bf16 terms a weight would have 16 bits, and the
// products with V twice as long.)
//
// Measured (GB300): 8192 tokens, 32 heads on 4 of 128: 310 us, 1.77 PFLOP/s (0.92 of the measured
// cuBLAS rate); 16 on 2 of 256: 272 to 284 us, 1.94 to 2.02 PFLOP/s; 4 prompts of 3000 to 4096 with a
// window of 1024: 151 us; 6 of 329 to 1993, 24 on 2 of 256: 95 to 112 us (one tile to a CTA: each chunk
// is 64 KB a CTA from L2, 9 TB/s over the GPU, and the time changes from process to process); 64 of 50 to
// 150: 38 to 41 us; one of 77: 7.1 us.  A chunk's turn of two
// tiles takes 3130 cycles of which its MMAs need 2048: from one tile's S to its next O pass S's
// commit (450 cycles until a warp sees it), the softmax (ld 180, maximum 500, weights 800) and P's
// arrival (300), and the other tile's products cover 1024 of that.  One tile with three S
// buffers and two or three groups of softmax warps takes fewer cycles (2 x 1380), but reads K and V
// twice as often, and at that load the clock falls (1.72 GHz instead of 2.07): 347 to 360 us.  Half rows on
// twice the softmax warps: 398; output warps of their own with Q in two buffers: 346; the maximum after the
// first weights and P in four parts: 388.  What counted: the output's stores in runs of 64 bytes
// (windowed 187 -> 169, 64 prompts of 50 to 150 71 -> 55), the MMA warp's loops rolled, units found by one
// role (170 -> 163, 55 -> 49), masks as words of bits (163 -> 150, 49 -> 42, long 316 -> 310).
//
// Roles in a CTA:
//   softmax   four warps a tile, a thread per vector: its row of S to registers, P = exp2(S c -
//             base) as bf16 over the columns it has read, 64 tokens at a time; at a unit's end O from
//             tensor memory to the output
//   copy      one warp: Q, K and V by TMA into a ring of stages
//   relay     one warp: tells the first CTA's MMA warp that a stage is there, and zeroes V rows
//             that no row of the unit sees (another sequence's, or what lies behind the last) and
//             elements that are not finite (see "Values that are not finite")
//   MMA       one warp of the first CTA.  At head_dim 128 two tiles take turns: O_0, S_0 of the next
//             chunk, O_1, S_1; at 256 one tile has two S buffers and S runs ahead.  Its code comes from far,
//             between the softmax warps' long loops, so its loops over MMAs are rolled
//
// Tensor memory (512 columns): S buffers at 0 and 128, O from 256.
// mbarriers, all waits bounded (2 s; a wait that gives up sets the status word):
//   full[s], free[s]   stage s copied (in each CTA); its MMAs complete (commit, to both)
//   ready[s]           stage s there in both CTAs (the first CTA's; one arrival of each relay)
//   qfull, qready, qfree   the same for Q
//   barS[y]            S buffer y complete (and with two tiles the tile's O of the chunk before)
//   pready[y][h]       half h of P in buffer y written (four warps of each CTA)
//   barO               O complete up to a chunk (one tile), partO[t]  at a unit's end
// A phase of a barrier is only told from its neighbours, so every waiter is at most one phase
// behind: barO is waited for only where barS has said that the phase before is complete, and
// a unit's end has a barrier of its own.
#include "qsa_tc_pair.cuh"

#include <cuda.h>

#include <algorithm>

namespace qsa {
namespace prompt {
namespace {

using namespace tc;

// Bounds-check codes (reported by bounds-checked builds only).
[[maybe_unused]] constexpr int kChkUnit = 0xD01;    // unit's rows out of range
[[maybe_unused]] constexpr int kChkOut = 0xD02;     // output row out of range

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNoBase = -1e30f;
constexpr float kHeadroom = 8.f;
constexpr int kTok = 128;              // tokens per chunk
constexpr int kUnits = 4;              // units in shared memory

struct Args {
  int B, Hq, Hkv, G, T;
  int rho;                 // rows of a tile
  int window;
  float c;                 // sm_scale log2(e)
  const int32_t* cu;       // [B + 1]
  const float* sinks;
  const __nv_bfloat16* v;  // as map_v has it; its row stride in elements
  long long v_stride;
  __nv_bfloat16* out;      // [T][Hq][D]
  float* lse;              // [T][Hq]
  int* status;
};

template <int D_>
struct PT {
  static constexpr int D = D_;
  static constexpr int kTiles = D == 128 ? 2 : 1;        // tiles of a CTA
  static constexpr int kSoft = 4 * kTiles;               // softmax warps
  static constexpr int kMma = kSoft, kCopy = kSoft + 1, kRelay = kSoft + 2;
  static constexpr int kThreads = 32 * (kSoft + 4);
  // Registers per thread after the roles part, of 168 at launch (two tiles); with one tile there
  // are enough for everybody.
  static constexpr int kSoftRegs = 216, kOtherRegs = 72;
  static_assert(32 * (8 * kSoftRegs + 4 * kOtherRegs) <= 384 * 168, "registers");
  static constexpr int kQBlk = 128 * 128;                // 64 dims of a tile's vectors
  static constexpr int kQBytes = 128 * D * 2;
  static constexpr int kStage = 128 * D;                 // 64 tokens of K, or D/2 dims of 128 tokens of V
  static constexpr int kStages = D == 128 ? 10 : 5;
  static constexpr int kKBlk = 64 * 128;                 // 64 dims of 64 tokens
  static constexpr int kVBlk = kTok * 128;               // 64 dims of 128 tokens
  static constexpr uint32_t kOCol = 256;
  static constexpr int kBars = 3 * kStages + 3 + 2 + 4 + 1 + 2 + 1 + kUnits;
  static constexpr int kSmem = 1024 + kTiles * kQBytes + kStages * kStage + kUnits * 32 + kBars * 8 + 16 + kUnits * 8;
  static_assert(kSmem <= 227 * 1024, "shared memory");
};

// ---- units -----------------------------------------------------------------------
struct Unit {
  int start, row0, rows;   // the sequence's first row; the unit's rows within it
  int kvh;
  int n_all, lo_all;       // tokens: past the last that its last row sees, first that its first row sees
  int chunks;              // of 128 tokens from lo_all on; 0: there is no unit more
};

// The units that the copy warp has found, for the other roles of its CTA.  (Each for itself, every
// role's units began with the search, and its code was there four times.)  A slot is written again
// when its readers are done with it: the copy warp finds unit i + 4 behind its copies of unit i + 3,
// which waited for unit i + 2's Q to be free, so that the MMA warp and both relays had come to unit i + 2 and
// the softmax warps to unit i + 1.
struct Units {
  int4* slots;             // [kUnits][2]
  uint64_t* there;         // [kUnits]
  int at;

  __device__ __forceinline__ void put(const Unit& u) {
    const int s = at % kUnits;
    if ((threadIdx.x & 31) == 0) {
      slots[2 * s] = make_int4(u.start, u.row0, u.rows, u.kvh);
      slots[2 * s + 1] = make_int4(u.n_all, u.lo_all, u.chunks, 0);
      ws_arrive(&there[s]);
    }
    __syncwarp();
    ++at;
  }
  // The next unit; false behind the last one and where the wait gave up (then dead is set).
  __device__ __forceinline__ bool next(Unit& u, bool& dead) {
    const int s = at % kUnits;
    if (gave_up(&there[s], at / kUnits)) {
      dead = true;
      return false;
    }
    u = before(at++);
    return u.chunks > 0;
  }
  // Unit `nth`, which the reader has come to and is not yet two units past.
  __device__ __forceinline__ Unit before(int nth) const {
    const int s = nth % kUnits;
    const int4 a = slots[2 * s], b = slots[2 * s + 1];
    return Unit{a.x, a.y, a.z, a.w, b.x, b.y, b.z};
  }
};

// ---- values that are not finite ----------------------------------------------------
// A weight of 0 times a V that is not finite is NaN: of a token that some rows of the unit see and
// others do not (from the second row's on, and those that the last row has left behind), such a value would
// reach rows that do not see it.  The relay takes these out of the tile and leaves a note; behind such a unit,
// rows get what the MMA left out, from V as it lies in memory.  The notes say for which unit (its number from 1
// on) rather than whether, so that nobody has to take them back; each of the pair's relays, which has half of the
// dims, leaves one in both CTAs, ahead of the arrival that lets the chunk's products begin. Only tokens of
// that kind are looked at, with one multiply-add for two elements: the relay's instructions are taken from the
// softmax warps' (64 prompts of 50 to 150 tokens, 32 heads on 4 of 128, 38.8 us without, 41.0 with; windowed 150.0
// and 150.6, a window of 64 49.8 and 49.8, long 307.5 and 307.6; the whole chunk, four instructions an element, 38.9 and
// 43.0, 150.0 and 156, 49.8 and 58).
struct Partly {            // tokens of the unit's sequence that not all of its rows see: those before `left`
  int left, right;         // and those from `right` on
  __device__ __forceinline__ Partly(const Unit& u, int window)
      : left(window > 0 ? u.n_all - window : 0), right(u.row0 + 1) {}
};
// Bits 15 and 31 for two bf16 that are not finite (the others are anything).
__device__ __forceinline__ uint32_t not_finite2(uint32_t w) { return (w & 0x7F807F80u) + 0x00800080u; }
__device__ __forceinline__ uint32_t not_finite8(const uint4& x) {
  return (not_finite2(x.x) | not_finite2(x.y) | not_finite2(x.z) | not_finite2(x.w)) & 0x80008000u;
}
// Zeros times eight bf16, added to `sum`: NaN from the first one on that is not finite.
__device__ __forceinline__ __nv_bfloat162 zeros_or_nan(const uint4& x, __nv_bfloat162 sum) {
  const __nv_bfloat162 zero = __float2bfloat162_rn(0.f);
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) sum = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&w[k]), zero, sum);
  return sum;
}
__device__ __forceinline__ uint32_t finite2(uint32_t w) {      // those as zeros
  return w & ~(((not_finite2(w) & 0x80008000u) >> 15) * 0xFFFFu);
}
__device__ __forceinline__ void note_both(uint32_t* at, uint32_t value) {
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, 0;\n\tst.shared::cluster.u32 [a], %1;\n\t"
      "mapa.shared::cluster.u32 a, %0, 1;\n\tst.shared::cluster.u32 [a], %1;\n\tfence.acq_rel.cluster;\n\t}" ::"r"(
          smem_u32(at)), "r"(value)
      : "memory");
}

// Adds to a row's output the values that are not finite of the tokens that it sees and other rows of the unit
// do not.  v: token 0 of the sequence.
template <int D>
__device__ __forceinline__ void add_not_finite(const Unit& u, int window, const __nv_bfloat16* v, long long stride, int lo,
                                               int n, __nv_bfloat16* out) {
  const Partly part(u, window);
#pragma unroll 1
  for (int d = 0; d < D; d += 8) {
    float add[8] = {};
    bool any = false;
#pragma unroll 1
    for (int t = lo; t < n; ++t) {
      if (t >= part.left && t < part.right) t = part.right;
      if (t >= n) break;
      const uint4 x = *reinterpret_cast<const uint4*>(v + t * stride + d);
      if (!not_finite8(x)) continue;
      any = true;
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t odd = w[k] & ~finite2(w[k]);
        add[2 * k] += __uint_as_float(odd << 16);
        add[2 * k + 1] += __uint_as_float(odd & 0xFFFF0000u);
      }
    }
    if (!any) continue;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (add[k] != 0.f) out[d + k] = __float2bfloat16_rn(__bfloat162float(out[d + k]) + add[k]);
  }
}

// Walks a worker's units; the copy warp's.  With up to 32 sequences a lane has one, and the
// units go by their number within their sequence, last (longest) first.  With more sequences
// the slots of a sequence begin at cu[b] / U + b, which leaves room for all its tiles (and some
// slots empty) and can be searched: units then go in their sequences' order (39 prompts of 100 tokens and one of
// 4096, 32 heads on 4 of 128: 106 us with the long one first, 111 with it last, 129 with it in the middle).
struct Walker {
  const Args& a;
  int U, worker, workers, turn;
  int start, n;            // lane b's sequence
  long long units;
  int most;                // tiles of the longest

  __device__ __forceinline__ Walker(const Args& a_, int unit_rows, int worker_, int workers_)
      : a(a_), U(unit_rows), worker(worker_), workers(workers_), turn(0) {
    const int lane = threadIdx.x & 31;
    start = n = most = 0;
    if (a.B <= 32) {
      if (lane < a.B) range(lane, start, n);
      const int tiles = (n + U - 1) / U;
      most = __reduce_max_sync(0xffffffffu, tiles);
      units = (long long)__reduce_add_sync(0xffffffffu, tiles) * a.Hkv;
    } else {
      units = ((long long)min(max(__ldg(a.cu + a.B), 0), a.T) / U + a.B) * a.Hkv;
    }
  }
  __device__ __forceinline__ void range(int b, int& first, int& rows) const {
    first = min(max(__ldg(a.cu + b), 0), a.T);
    rows = max(min(__ldg(a.cu + b + 1), a.T) - first, 0);
  }
  __device__ __forceinline__ bool next(Unit& u) {
    const int lane = threadIdx.x & 31;
    while (true) {
      const long long at = (long long)turn * workers + ((turn & 1) ? workers - 1 - worker : worker);
      if ((long long)turn * workers >= units) return false;
      ++turn;
      if (at >= units) continue;
      const int slot = (int)(at / a.Hkv);
      u.kvh = (int)(at - (long long)slot * a.Hkv);
      int tile, rows;      // the unit's number within its sequence, the sequence's rows
      if (a.B <= 32) {
        // the largest i with more than `slot` tiles numbered i or higher
        const int tiles = (n + U - 1) / U;
        int lo = 0, hi = most;
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if ((int)__reduce_add_sync(0xffffffffu, max(tiles - mid, 0)) > slot) lo = mid;
          else hi = mid;
        }
        tile = lo;
        const int nth = slot - (int)__reduce_add_sync(0xffffffffu, max(tiles - tile - 1, 0));
        const uint32_t have = __ballot_sync(0xffffffffu, tiles > tile);
        // (of the sequences that have such a tile, the nth)
        const uint32_t mine = __ballot_sync(0xffffffffu, tiles > tile && __popc(have & ((1u << lane) - 1u)) == nth);
        const int b = __ffs(mine) - 1;
        u.start = __shfl_sync(0xffffffffu, start, b);
        rows = __shfl_sync(0xffffffffu, n, b);
      } else {
        int lo = 0, hi = a.B;
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (min(max(__ldg(a.cu + mid), 0), a.T) / U + mid <= slot) lo = mid;
          else hi = mid;
        }
        range(lo, u.start, rows);
        tile = slot - (min(max(__ldg(a.cu + lo), 0), a.T) / U + lo);
        if (tile < 0 || tile >= (rows + U - 1) / U) continue;
        tile = (rows + U - 1) / U - 1 - tile;
      }
      u.row0 = tile * U;
      u.rows = min(U, rows - u.row0);
      if (!QSA_IN_BOUNDS(u.row0 >= 0 && u.rows > 0 && u.start + rows <= a.T, kChkUnit)) continue;
      u.n_all = u.row0 + u.rows;
      u.lo_all = a.window > 0 ? max(u.row0 + 1 - a.window, 0) : 0;
      u.chunks = (u.n_all - u.lo_all + kTok - 1) / kTok;
      return true;
    }
  }
};

__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];"
      ::"r"(dst), "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <int D>
__global__ void __launch_bounds__(PT<D>::kThreads, 1)
prompt_kernel(const __grid_constant__ Args a, const __grid_constant__ CUtensorMap map_q,
              const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v) {
  using T = PT<D>;
  constexpr int kTiles = T::kTiles, CG = 2;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)(blockIdx.x & 1);                // CTA of the pair
  const int worker = (int)(blockIdx.x >> 1), workers = (int)(gridDim.x >> 1);

  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem;                                    // [kTiles][kQBytes]
  uint8_t* ring = sQ + kTiles * T::kQBytes;              // [kStages][kStage]
  int4* s_units = reinterpret_cast<int4*>(ring + T::kStages * T::kStage);
  uint64_t* full = reinterpret_cast<uint64_t*>(s_units + 2 * kUnits);
  uint64_t* free_ = full + T::kStages;
  uint64_t* ready = free_ + T::kStages;
  uint64_t* qfull = ready + T::kStages;
  uint64_t* qready = qfull + 1;
  uint64_t* qfree = qfull + 2;
  uint64_t* barS = qfull + 3;                            // [2]
  uint64_t* pready = barS + 2;                           // [buffer][half]
  uint64_t* barO = pready + 4;
  uint64_t* partO = barO + 1;                            // [2]
  uint64_t* mdone = partO + 2;                           // after a give-up: every MMA issued has completed
  uint64_t* uthere = mdone + 1;                          // [kUnits]
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(uthere + kUnits);
  uint32_t* s_odd = s_tmem + 4;                          // [kUnits][CTA]: number of a unit with V that is not finite

  if (tid == 0) {
    for (int s = 0; s < T::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&free_[s], 1);
      mbar_init(&ready[s], CG);
    }
    mbar_init(qfull, 1);
    mbar_init(qready, CG);
    mbar_init(qfree, 1);
    for (int x = 0; x < 2; ++x) {
      mbar_init(&barS[x], 1);
      mbar_init(&pready[2 * x], 4 * CG);
      mbar_init(&pready[2 * x + 1], 4 * CG);
      mbar_init(&partO[x], 1);
    }
    for (int s = 0; s < kUnits; ++s) mbar_init(&uthere[s], 1);
    mbar_init(barO, 1);
    mbar_init(mdone, 1);
    s_tmem[1] = 0u;   // set when a CTA of the pair gave up
    for (int i = 0; i < 2 * kUnits; ++i) s_odd[i] = 0u;
    fence_mbar_init();
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(s_tmem)),
                 "r"(512u));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  tc_fence_before();
  cluster_sync();                                        // the pair's barriers are initialised
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  pdl_wait();
  pdl_trigger();
  const int unit_rows = 2 * kTiles * a.rho;
  bool dead = false;
  Units units{s_units, uthere, 0};

  if (warp < T::kSoft) {
    // ==== softmax ==================================================================
    if constexpr (kTiles == 2) regs_up<T::kSoftRegs>();
    const int t = warp >> 2, row = tid & 127;
    const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t tO = tmem + T::kOCol + t * D + lane_off;
    const int my_row = (t * CG + rank) * a.rho + row / a.G;       // within the unit
    const int my_head = row % a.G;
    const bool in_tile = row < a.rho * a.G;
    int chunks = 0, s_waits = 0, parts = 0;     // chunks, waits on barS (two tiles), units so far
    Unit u;
    bool more = units.next(u, dead);
    while (!dead && more) {
      const bool real = in_tile && my_row < u.rows;
      const int n = real ? u.row0 + my_row + 1 : 0;
      const int lo = a.window > 0 ? max(n - a.window, 0) : 0;
      const int head = u.kvh * a.G + my_head;
      const size_t orow = ((size_t)u.start + u.row0 + my_row) * a.Hq + head;
      // of the warp's vectors: where its first row ends, where its last row's window begins
      const int n_least = __reduce_min_sync(0xffffffffu, real ? n : 0x7FFFFFFF);
      const int lo_most = __reduce_max_sync(0xffffffffu, real ? lo : 0);
      const bool some = __any_sync(0xffffffffu, real);   // (a warp without a row only keeps step)
      float base = kNoBase;
      RowSum sum;
      const int unit_chunks = u.chunks, lo_all = u.lo_all;
      for (int c = 0; c < unit_chunks; ++c, ++chunks) {
        const int y = kTiles == 2 ? t : chunks & 1;      // S buffer
        const uint32_t tS = tmem + y * kTok + lane_off;
        const int tok0 = lo_all + c * kTok;
        if (gave_up(&barS[y], kTiles == 2 ? s_waits : chunks >> 1)) { dead = true; break; }
        ++s_waits;
        tc_fence_after();
        if (!some) {
          tc_fence_before();
          warp_arrive<CG>(&pready[2 * y]);
          warp_arrive<CG>(&pready[2 * y + 1]);
          continue;
        }
        // The row's logits, those it does not see at -inf.
        float z[kTok];
#pragma unroll
        for (int i = 0; i < kTok / 32; ++i) tmem_ld32(tS + 32 * i, z + 32 * i);
        tmem_wait_ld_of(z);
        if (tok0 + kTok > n_least || tok0 < lo_most) {
          // (a word of bits for 32 tokens: a third of the code that two comparisons a token take)
          const int end = n - tok0, begin = lo - tok0;
          auto below = [](int x) { return x >= 32 ? 0xFFFFFFFFu : x <= 0 ? 0u : (1u << x) - 1u; };
#pragma unroll
          for (int w = 0; w < kTok / 32; ++w) {
            const uint32_t sees = below(end - 32 * w) & ~below(begin - 32 * w);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!((sees >> i) & 1u)) z[32 * w + i] = -INFINITY;
          }
        }
        float m8[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) m8[i] = z[i];
#pragma unroll
        for (int i = 8; i < kTok; i += 2) m8[(i >> 1) & 7] = fmax3(m8[(i >> 1) & 7], z[i], z[i + 1]);
        const float top = a.c * fmax3(fmax3(m8[0], m8[1], m8[2]), fmax3(m8[3], m8[4], m8[5]), fmaxf(m8[6], m8[7]));
        const bool moves = top > base + kHeadroom;
        if (__any_sync(0xffffffffu, moves)) {
          const float nb = moves ? top : base;
          const float alpha = exp2_approx(base - nb);
          base = nb;
          sum.scale(alpha);
          if (c > 0) {
            // with two tiles barS has said that O is complete up to the chunk before
            if (kTiles == 1 && gave_up(barO, chunks - 1)) { dead = true; break; }
            tc_fence_after();
#pragma unroll 1
            for (int i = 0; i < D / 16; ++i) {
              float o16[16];
              tmem_ld16(tO + 16 * i, o16);
              tmem_wait_ld_of(o16);
#pragma unroll
              for (int k = 0; k < 16; ++k) o16[k] *= alpha;
              tmem_st16(tO + 16 * i, o16);
            }
          }
        }
        // P, 64 tokens at a time, over the first columns they were read from.
        const float2 c2 = make_float2(a.c, a.c), b2 = make_float2(-base, -base);
        float2 part = make_float2(0.f, 0.f);               // the chunk's weights
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int k = 64 * h + 32 * q + 2 * i;
              const float2 x = fma2(make_float2(z[k], z[k + 1]), c2, b2);
              const float2 e = make_float2(exp2_approx(x.x), exp2_approx(x.y));
              part = add2(part, e);
              pk[i] = pack_bf16(e.x, e.y);
            }
            tmem_st16u(tS + 32 * h + 16 * q, pk);
          }
          tmem_wait_st();
          tc_fence_before();
          warp_arrive<CG>(&pready[2 * y + h]);
        }
        sum.add(part);
      }
      if (dead) break;
      // ---- the unit's output, the next unit found meanwhile ------------------------------
      more = units.next(u, dead);
      if (dead || gave_up(&partO[t], parts)) { dead = true; break; }
      ++parts;
      tc_fence_after();
      float l = sum.total(), f = 1.f;
      if (a.sinks && real) {
        const float s2 = a.sinks[head] * kLog2e, nm = fmaxf(base, s2);
        f = exp2_approx(base - nm);
        l = l * f + exp2_approx(s2 - nm);
        base = nm;
      }
      const float r = f / l;                             // (a row sees itself at least)
      const bool store = real && QSA_IN_BOUNDS(orow < (size_t)a.T * a.Hq, kChkOut);
      uint32_t row4[4], rows4 = 0u;                      // the rows of this lane and its three neighbours (below 2^32)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        row4[k] = __shfl_sync(0xffffffffu, (uint32_t)orow, (lane & 28) + k);
        rows4 |= (uint32_t)__shfl_sync(0xffffffffu, (int)store, (lane & 28) + k) << k;
      }
#pragma unroll 1
      for (int d0 = 0; d0 < D && some; d0 += 32) {
        float o32[32];
        tmem_ld32(tO + d0, o32);
        tmem_wait_ld_of(o32);
        uint32_t w[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) w[k] = pack_bf16(o32[2 * k] * r, o32[2 * k + 1] * r);
        transpose4(w, lane);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (rows4 >> k & 1u)
            *reinterpret_cast<uint4*>(a.out + (size_t)row4[k] * D + d0 + 8 * (lane & 3)) =
                make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
      }
      if (store) a.lse[orow] = (base + log2f(l)) * kLn2;
      const uint2 odd = *reinterpret_cast<const uint2*>(s_odd + 2 * ((parts - 1) % kUnits));
      if (__builtin_expect(odd.x == (uint32_t)parts || odd.y == (uint32_t)parts, false)) {
        const Unit was = units.before(parts - 1);
        __syncwarp();                                    // (the row was stored by its neighbours)
        if (store)
          add_not_finite<D>(was, a.window, a.v + was.start * a.v_stride + was.kvh * D, a.v_stride, lo, n,
                            a.out + orow * D);
      }
    }
  } else {
    if constexpr (kTiles == 2) regs_down<T::kOtherRegs>();
    Unit u;
    int pos = 0, parts = 0;                              // stages so far (two per chunk), units
    if (warp == T::kCopy) {
      // ==== copies =================================================================
      const uint32_t q_bytes = (uint32_t)(kTiles * (D / 64) * 128 * a.rho * a.G);
      Walker walk(a, unit_rows, worker, workers);
      while (!dead && walk.next(u)) {
        units.put(u);
        for (int c = 0; c < u.chunks && !dead; ++c) {
          const int tok = u.start + u.lo_all + c * kTok;
#pragma unroll 1
          for (int v = 0; v < 2; ++v, ++pos) {
            const int s = pos % T::kStages, use = pos / T::kStages;
            if (use > 0 && gave_up(&free_[s], use - 1)) { dead = true; break; }
            if (lane == 0) {
              const uint32_t to = smem_u32(ring + s * T::kStage);
              mbar_arrive_expect_tx(&full[s], T::kStage);
              if (v) {
#pragma unroll
                for (int x = 0; x < D / 128; ++x)
                  tma_load(to + x * T::kVBlk, &map_v, rank * (D / 2) + 64 * x, u.kvh, tok, &full[s]);
              } else {
#pragma unroll
                for (int x = 0; x < D / 64; ++x)
                  tma_load(to + x * T::kKBlk, &map_k, 64 * x, u.kvh, tok + 64 * rank, &full[s]);
              }
            }
            __syncwarp();
          }
          if (c == 0 && !dead) {
            if (parts > 0 && gave_up(qfree, parts - 1)) { dead = true; break; }
            if (lane == 0) {
              mbar_arrive_expect_tx(qfull, q_bytes);
#pragma unroll 1
              for (int t = 0; t < kTiles; ++t)
#pragma unroll
                for (int x = 0; x < D / 64; ++x)
                  tma_load(smem_u32(sQ + t * T::kQBytes + x * T::kQBlk), &map_q, 64 * x, u.kvh * a.G,
                           u.start + u.row0 + (t * CG + rank) * a.rho, qfull);
            }
            __syncwarp();
            ++parts;
          }
        }
      }
      if (!dead) units.put(Unit{});
      // Nothing may still be on its way when the block ends, whoever gave up.
#pragma unroll 1
      for (int s = 0; s < T::kStages; ++s) {
        const int uses = pos / T::kStages + (s < pos % T::kStages ? 1 : 0);
        if (uses > 0 && gave_up(&full[s], uses - 1)) dead = true;
      }
      if (parts > 0 && gave_up(qfull, parts - 1)) dead = true;
      // Nor may an arrival of the MMAs' commits that nobody else waits for: the softmax warps wait for a unit's
      // last products, not for the barriers that are told of them next.  A lane waits for each.
      if (!dead) {
        static_assert(T::kStages + 2 <= 32, "lanes");
        const bool stage = lane < T::kStages, o = lane == T::kStages + 1;
        uint64_t* bar = stage ? &free_[lane] : o ? barO : qfree;
        const int last = stage ? (pos - 1 - lane) / T::kStages : o ? pos / 2 - 1 : parts - 1;
        dead = lanes_gave_up(bar, last, stage ? lane < pos : o ? kTiles == 1 && pos > 0 : lane == T::kStages && parts > 0);
      }
    } else if (warp == T::kRelay) {
      // ==== relay ====================================================================
      // Q of the first unit as soon as it is there (S waits for it), of the others, which follows the last S of
      // the unit before, behind V, which has long been there.
      auto q_relayed = [&]() {
        if (gave_up(qfull, parts)) dead = true;
        else warp_arrive<CG>(qready);
        ++parts;
        return !dead;
      };
      while (!dead && units.next(u, dead)) {
        const int nth = units.at;                        // from 1 on
        const Partly part(u, a.window);
        for (int c = 0; c < u.chunks && !dead; ++c) {
          const int tok0 = u.lo_all + c * kTok;
#pragma unroll 1
          for (int v = 0; v < 2; ++v, ++pos) {
            const int s = pos % T::kStages, use = pos / T::kStages;
            if (v && nth == 1 && c == 0 && !q_relayed()) break;
            if (gave_up(&full[s], use)) { dead = true; break; }
            if (v && (tok0 + kTok > part.right || tok0 < part.left)) {
              uint4* tile = reinterpret_cast<uint4*>(ring + s * T::kStage);
              // rows of V that no vector of the unit sees may hold anything; 0 keeps 0 x V at 0
              for (int x = 8 * max(u.n_all - tok0, 0) + lane; x < 8 * kTok; x += 32)
#pragma unroll
                for (int i = 0; i < T::kStage / T::kVBlk; ++i)
                  tile[i * (T::kVBlk / 16) + x] = make_uint4(0u, 0u, 0u, 0u);
              __nv_bfloat162 odd = __float2bfloat162_rn(0.f);
#pragma unroll 1
              for (int side = 0; side < 2; ++side) {
                const int from = side ? max(part.right - tok0, 0) : 0;
                const int to = min(side ? u.n_all : min(part.left, part.right), tok0 + kTok) - tok0;
#pragma unroll 4
                for (int x = 8 * from + lane; x < 8 * to; x += 32)
#pragma unroll
                  for (int i = 0; i < T::kStage / T::kVBlk; ++i) odd = zeros_or_nan(tile[i * (T::kVBlk / 16) + x], odd);
              }
              if (__any_sync(0xffffffffu, __hisnan(odd.x) || __hisnan(odd.y))) {
#pragma unroll 1
                for (int x = lane; x < T::kStage / 16; x += 32) {
                  const int tok = tok0 + ((x >> 3) & (kTok - 1));
                  const uint4 y = tile[x];
                  if (tok < part.left || tok >= part.right)
                    tile[x] = make_uint4(finite2(y.x), finite2(y.y), finite2(y.z), finite2(y.w));
                }
                if (lane == 0) note_both(&s_odd[2 * ((nth - 1) % kUnits) + rank], (uint32_t)nth);
              }
              fence_proxy_async_smem();
            }
            warp_arrive<CG>(&ready[s]);
          }
          if (nth > 1 && c == 0 && !dead) q_relayed();
        }
      }
    } else if (warp == T::kMma && rank == 0) {
      // ==== MMA issue ================================================================
      const uint32_t one = elect_one();
      constexpr uint32_t kBf16 = (1u << 7) | (1u << 10);   // instruction descriptor: bf16 A and B
      const uint32_t id_s = f16_idesc(256, kTok) | kBf16, id_o = f16_idesc(256, D) | kBf16 | kIdescBMn;
      int chunk = 0;                                       // chunks of earlier units
      const uint32_t q_lo = (uint32_t)sw128_desc(smem_u32(sQ)), r_lo = (uint32_t)sw128_desc(smem_u32(ring));
      const uint32_t v_lo = (uint32_t)sw128_mn_desc(smem_u32(ring), T::kVBlk);
      constexpr uint64_t kHi = (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
      auto slot_k = [&](int n) { return (2 * n) % T::kStages; };
      auto slot_v = [&](int n) { return (2 * n + 1) % T::kStages; };
      auto there = [&](int p) {                            // waits for the stage at position p
        const bool ok = !gave_up(&ready[p % T::kStages], p / T::kStages);
        tc_fence_after();
        return ok;
      };
      auto issue_s = [&](int t, int y, int n) {
        uint32_t dq = q_lo + t * (T::kQBytes >> 4), dk = r_lo + slot_k(n) * (T::kStage >> 4);
#pragma unroll 1
        for (int x = 0; x < D / 64; ++x) {
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            mma_ss<CG>(one, tmem + y * kTok, kHi | (dq + 2 * ks), kHi | (dk + 2 * ks), id_s, (x | ks) ? 1u : 0u);
          dq += T::kQBlk >> 4;
          dk += T::kKBlk >> 4;
        }
      };
      auto issue_o = [&](int t, int y, int n, int h, bool first) {   // 64 tokens
        const uint32_t dv = v_lo + slot_v(n) * (T::kStage >> 4) + 512 * h;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          mma_ts<CG>(one, tmem + T::kOCol + t * D, tmem + y * kTok + 32 * h + 8 * ks, kHi | (dv + 128 * ks), id_o,
                     (first && ks == 0) ? 0u : 1u);
      };
      while (!dead && units.next(u, dead)) {
        const int C = u.chunks;
        if (gave_up(qready, parts) || !there(2 * chunk)) { dead = true; break; }
        ++parts;
        if constexpr (kTiles == 2) {
          issue_s(0, 0, chunk);
          commit<CG>(one, &barS[0]);
          issue_s(1, 1, chunk);
          commit<CG>(one, &barS[1]);
          commit<CG>(one, &free_[slot_k(chunk)]);
          if (C == 1) commit<CG>(one, qfree);
          // (the stages of a chunk are waited for while the products before it run)
          if (!there(2 * chunk + 1) || (C > 1 && !there(2 * chunk + 2))) { dead = true; break; }
          for (int c = 0; c < C && !dead; ++c) {
            const int n = chunk + c;
            const bool more = c + 1 < C;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                if (gave_up(&pready[2 * t + h], n)) { dead = true; break; }
                tc_fence_after();
                issue_o(t, t, n, h, c == 0 && h == 0);
              }
              if (dead) break;
              if (more) {
                issue_s(t, t, n + 1);
                commit<CG>(one, &barS[t]);
              } else {
                commit<CG>(one, &partO[t]);
              }
            }
            if (dead) break;
            commit<CG>(one, &free_[slot_v(n)]);
            if (more) {
              commit<CG>(one, &free_[slot_k(n + 1)]);
              if (c + 2 == C) commit<CG>(one, qfree);
              if (!there(2 * n + 3) || (c + 2 < C && !there(2 * n + 4))) { dead = true; break; }
            }
          }
        } else {
          for (int c = 0; c < 2 && c < C; ++c) {
            const int n = chunk + c;
            if (c > 0 && !there(2 * n)) { dead = true; break; }
            issue_s(0, n & 1, n);
            commit<CG>(one, &barS[n & 1]);
            commit<CG>(one, &free_[slot_k(n)]);
            if (c + 1 == C) commit<CG>(one, qfree);
          }
          for (int c = 0; c < C && !dead; ++c) {
            const int n = chunk + c, y = n & 1;
            if (!there(2 * n + 1)) { dead = true; break; }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (gave_up(&pready[2 * y + h], n >> 1)) { dead = true; break; }
              tc_fence_after();
              issue_o(0, y, n, h, c == 0 && h == 0);
            }
            if (dead) break;
            commit<CG>(one, &free_[slot_v(n)]);
            commit<CG>(one, barO);
            if (c + 1 == C) commit<CG>(one, &partO[0]);
            if (c + 2 < C) {
              if (!there(2 * n + 4)) { dead = true; break; }
              issue_s(0, y, n + 2);
              commit<CG>(one, &barS[y]);
              commit<CG>(one, &free_[slot_k(n + 2)]);
              if (c + 3 == C) commit<CG>(one, qfree);
            }
          }
        }
        chunk += C;
      }
    }
  }

  // As in the tile kernel (qsa_dense_tile.cu): every MMA has completed where nothing gave up;
  // after a give-up, wait for what the MMA warp issued before its memory goes.
  if (dead) atomicExch(a.status, kStatusWaitTimeout);
  tc_fence_before();
  bool any_dead = __syncthreads_or(dead);
  if (any_dead && tid == 0)
    asm volatile(
        "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, 0;\n\tst.shared::cluster.u32 [a], %1;\n\t"
        "mapa.shared::cluster.u32 a, %0, 1;\n\tst.shared::cluster.u32 [a], %1;\n\t}" ::"r"(smem_u32(s_tmem + 1)),
        "r"(1u)
        : "memory");
  cluster_sync();
  any_dead = s_tmem[1] != 0u;
  tc_fence_after();
  if (any_dead) {
    if (warp == T::kMma && rank == 0) commit<CG>(elect_one(), mdone);
    gave_up(mdone, 0);
    __syncthreads();
  }
  cluster_sync();
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encoder() {
  static const EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}

// Rows of `heads` heads of D elements, `stride` elements apart, in boxes of 64 dims x `box_heads` x `box_rows`.
bool encode(CUtensorMap* map, const void* p, int D, int heads, long long rows, long long stride, int box_heads,
            int box_rows) {
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows}, ones[3] = {1, 1, 1};
  return encoder()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), dims, strides, box, ones,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch(const Args& a, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                   cudaStream_t stream) {
  using T = PT<D>;
  auto* kern = prompt_kernel<D>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, T::kSmem);
  if (e != cudaSuccess) return e;
  // as many pairs as there can be units: every sequence's last may be a short one
  const long long unit_rows = 2 * T::kTiles * a.rho;
  const long long units = ((long long)a.T / unit_rows + std::min(a.B, a.T)) * a.Hkv;
  const long long pairs = std::min<long long>(sm_count() / 2, std::max<long long>(units, 1));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * pairs));
  cfg.blockDim = dim3(T::kThreads);
  cfg.dynamicSmemBytes = T::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, a, q, k, v);
}

}  // namespace
}  // namespace prompt

cudaError_t launch_prompt(const Geom& g, const PromptArgs& p, cudaStream_t stream) {
  if (!prompt::encoder()) return cudaErrorNotSupported;
  prompt::Args a = {};
  a.B = g.B;
  a.Hq = g.Hq;
  a.Hkv = g.Hkv;
  a.G = g.Hq / g.Hkv;
  a.T = (int)p.rows;
  a.rho = 128 / a.G;
  a.window = p.window;
  a.c = (float)std::min((double)p.sm_scale * 1.4426950408889634, 3e38);
  a.cu = p.cu;
  a.sinks = p.sinks;
  a.v = reinterpret_cast<const __nv_bfloat16*>(p.v);
  a.v_stride = p.v_stride;
  a.out = reinterpret_cast<__nv_bfloat16*>(p.out);
  a.lse = p.lse;
  a.status = reinterpret_cast<int*>(p.workspace);
  CUtensorMap q, k, v;
  if (!prompt::encode(&q, p.q, g.D, g.Hq, p.rows, p.q_stride, a.G, a.rho) ||
      !prompt::encode(&k, p.k, g.D, g.Hkv, p.rows, p.k_stride, 1, 64) ||
      !prompt::encode(&v, p.v, g.D, g.Hkv, p.rows, p.v_stride, 1, 128))
    return cudaErrorInvalidValue;
  return g.D == 256 ? prompt::launch<256>(a, q, k, v, stream) : prompt::launch<128>(a, q, k, v, stream);
}

}  // namespace qsa

QSA_BOUNDS_READER(bounds_word_prompt)
