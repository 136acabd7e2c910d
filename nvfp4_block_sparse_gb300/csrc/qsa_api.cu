// qsa_api.cu -- the library's C ABI (declared in include/qsa.h): host-side
// argument validation, the sm_103 gate and the launches on the caller's
// stream.  Nothing here allocates, synchronises (except the diagnostic
// qsa_workspace_status) or reads device data.
//
// TensorRT-LLM PR #20937 ("GB300 perf work on
// qwen3_8_flash_next_nvfp4__sm_103__tp1"), review of the grouped-verify
// tests: the grouped NVFP4 path runs on SM 10.3 only; callers pass their own
// buffers (Per-File QA: caller-provided buffers).
#include "qsa_common.cuh"

#include <math.h>
#include <stdint.h>

#include <atomic>

namespace {

using qsa::Geom;

constexpr unsigned long long kDefaultWaitNs = 2000000000ull;
std::atomic<unsigned long long> g_wait_ns{kDefaultWaitNs};

constexpr int64_t kMaxPackedRows = 1LL << 24;   // rows of all requests of a call, as B R

bool positive(double x) { return x > 0.0 && isfinite(x); }

// A number as the unevaluated sum of two doubles, about 100 bits: a rotation plan's frequencies
// are multiplied by positions up to 2^31, so 53 bits would show in the angle.
struct Two {
  double hi, lo;
};
Two two_sum(double a, double b) {
  const double s = a + b, v = s - a;
  return {s, (a - (s - v)) + (b - v)};
}
Two joined(double a, double b) {   // |a| >= |b|
  const double s = a + b;
  return {s, b - (s - a)};
}
Two operator+(Two a, Two b) {
  const Two s = two_sum(a.hi, b.hi), t = two_sum(a.lo, b.lo);
  const Two u = joined(s.hi, s.lo + t.hi);
  return joined(u.hi, u.lo + t.lo);
}
Two operator-(Two a, Two b) { return a + Two{-b.hi, -b.lo}; }
Two operator*(Two a, Two b) {
  const double p = a.hi * b.hi;
  return joined(p, fma(a.hi, b.hi, -p) + (a.hi * b.lo + a.lo * b.hi));
}
Two operator/(Two a, Two b) {
  const double q = a.hi / b.hi;
  const Two r = a - b * Two{q, 0.0};
  const double q2 = r.hi / b.hi;
  const Two r2 = r - b * Two{q2, 0.0};
  return joined(q, q2) + Two{r2.hi / b.hi, 0.0};
}
constexpr Two kTurnsPerRadian = {0x1.45f306dc9c883p-3, -0x1.6b01ec5417056p-57};   // 1 / (2 pi)

// theta^(-1/n): the rounded one, improved by Newton's steps on theta r^n = 1.
Two root(double theta, int n) {
  Two r = {pow(theta, -1.0 / n), 0.0};
  for (int step = 0; step < 2; ++step) {
    Two p = {theta, 0.0};
    for (int i = 0; i < n; ++i) p = p * r;
    const Two d = Two{1.0, 0.0} - p;
    r = r + Two{r.hi * (d.hi / n), 0.0};
  }
  return r;
}

// The fraction of a number of turns, in 2^-64 turns, to nearest.
uint64_t turn_fraction(Two t) {
  t = t - Two{floor(t.hi), 0.0};   // whole turns change nothing
  if (t.hi < 0.0) t = t + Two{1.0, 0.0};
  const double a = ldexp(t.hi, 64), whole = floor(a);
  const double rest = floor((a - whole) + ldexp(t.lo, 64) + 0.5);
  return (whole < 0x1p64 ? (uint64_t)whole : 0u) + (uint64_t)(int64_t)rest;
}

// The checks of a rotation's configuration.
qsa_status_t check_rope_config(const qsa_rope_config_t* config) {
  if (!config) return QSA_ERR_INVALID_ARG;
  const qsa_rope_config_t& c = *config;
  if (c.rotary_dim < 16 || c.rotary_dim > 2 * QSA_ROPE_MAX_PAIRS || c.rotary_dim % 16 != 0)
    return QSA_ERR_INVALID_ARG;
  if (c.scaling < QSA_ROPE_PLAIN || c.scaling > QSA_ROPE_WAVELENGTH) return QSA_ERR_INVALID_ARG;
  if (!(c.theta > 1.0) || !isfinite(c.theta)) return QSA_ERR_INVALID_ARG;
  if (!(c.attention_factor >= 0.0) || !isfinite(c.attention_factor)) return QSA_ERR_INVALID_ARG;
  const bool banded = c.scaling == QSA_ROPE_YARN || c.scaling == QSA_ROPE_WAVELENGTH;
  if (c.scaling != QSA_ROPE_PLAIN && !positive(c.factor)) return QSA_ERR_INVALID_ARG;
  if (banded && (!positive(c.original_context) || !positive(c.low) || !positive(c.high) ||
                 !(c.low < c.high)))
    return QSA_ERR_INVALID_ARG;
  return QSA_OK;
}

// The scaled frequencies of `pairs` pairs, as turns per position.
qsa_status_t spectrum(const qsa_rope_config_t& c, int pairs, uint64_t* out) {
  const double two_pi = 6.283185307179586476925;
  const bool banded = c.scaling == QSA_ROPE_YARN || c.scaling == QSA_ROPE_WAVELENGTH;
  // YARN: the dims that turn `high` and `low` times within the original context
  double first = 0.0, last = 1.0;
  if (c.scaling == QSA_ROPE_YARN) {
    const double per = 2 * pairs / (2.0 * log(c.theta));
    first = fmax(floor(per * log(c.original_context / (c.high * two_pi))), 0.0);
    last = fmin(ceil(per * log(c.original_context / (c.low * two_pi))), 2 * pairs - 1.0);
    last = fmax(last, first + 1e-3);
  }
  const Two one = {1.0, 0.0}, factor = {c.factor, 0.0}, r = root(c.theta, pairs);
  Two plain = one;
  for (int i = 0; i < pairs; ++i, plain = plain * r) {
    Two f = plain;
    if (c.scaling == QSA_ROPE_LINEAR) {
      f = f / factor;
    } else if (banded) {
      Two m;   // the scaled frequency's share
      if (c.scaling == QSA_ROPE_YARN) {
        m = Two{i - first, 0.0} / Two{last - first, 0.0};
      } else {
        const Two turns = Two{c.original_context, 0.0} * f * kTurnsPerRadian;
        m = one - (turns - Two{c.low, 0.0}) / two_sum(c.high, -c.low);
      }
      if (!(m.hi > 0.0)) m = {0.0, 0.0};
      if (m.hi >= 1.0) m = one;
      f = f * (one - m) + f / factor * m;
    }
    if (!(f.hi < 0x1p32)) return QSA_ERR_INVALID_ARG;
    out[i] = turn_fraction(f * kTurnsPerRadian);
  }
  return QSA_OK;
}

// A plan's other fields.
qsa_status_t finish_plan(const qsa_rope_config_t& c, qsa_rope_t* plan) {
  double amplitude = c.attention_factor;
  if (amplitude == 0.0)
    amplitude = c.scaling == QSA_ROPE_YARN && c.factor > 1.0 ? 0.1 * log(c.factor) + 1.0 : 1.0;
  plan->amplitude = (float)amplitude;
  plan->rotary_dim = c.rotary_dim;
  return positive(plan->amplitude) ? QSA_OK : QSA_ERR_INVALID_ARG;
}

bool plan_ok(const qsa_rope_t& rope) {
  return rope.rotary_dim >= 16 && rope.rotary_dim <= 2 * QSA_ROPE_MAX_PAIRS &&
         rope.rotary_dim % 16 == 0 && positive(rope.amplitude);
}

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// max_rows: 8 for the decode / verify attention and the rollback; the index
// scores, the selection, the prologue and the context row-tile attention also
// take long context row groups.
qsa_status_t check_geom(const qsa_geom_t* g, int max_rows = qsa::kMaxRows) {
  if (!g) return QSA_ERR_INVALID_ARG;
  if (g->batch < 1 || g->batch > 65535) return QSA_ERR_INVALID_ARG;
  if (g->rows_per_req < 1) return QSA_ERR_INVALID_ARG;
  if (g->num_q_heads < 1 || g->num_kv_heads < 1) return QSA_ERR_INVALID_ARG;
  if (g->num_q_heads % g->num_kv_heads != 0) return QSA_ERR_INVALID_ARG;
  if (g->max_blocks < 1 || g->num_pages < 1) return QSA_ERR_INVALID_ARG;
  // head_dim 128 with 64/128-token pages; head_dim 256 (PR #20276, Performance,
  // shared code touched: the target's 24 q / 2 KV heads at head_dim 256) with
  // 32-token pages (Known limitations: tokens_per_block 32) or 64.
  if (g->index_dim != qsa::kIndexDim) return QSA_ERR_UNSUPPORTED;
  if (g->head_dim == 128) {
    if (g->page_size != 64 && g->page_size != 128) return QSA_ERR_UNSUPPORTED;
  } else if (g->head_dim == 256) {
    if (g->page_size != 32 && g->page_size != 64) return QSA_ERR_UNSUPPORTED;
  } else {
    return QSA_ERR_UNSUPPORTED;
  }
  if (g->rows_per_req > max_rows) return QSA_ERR_UNSUPPORTED;
  if (g->num_q_heads > qsa::kMaxQHeads) return QSA_ERR_UNSUPPORTED;
  if (g->max_blocks > qsa::kMaxBlocks) return QSA_ERR_UNSUPPORTED;
  if ((long long)g->batch * g->rows_per_req > (1LL << 24)) return QSA_ERR_UNSUPPORTED;
  return QSA_OK;
}

Geom to_geom(const qsa_geom_t* g) {
  Geom r;
  r.B = g->batch;
  r.R = g->rows_per_req;
  r.Hq = g->num_q_heads;
  r.Hkv = g->num_kv_heads;
  r.D = g->head_dim;
  r.Di = g->index_dim;
  r.P = g->page_size;
  r.MB = g->max_blocks;
  r.NP = g->num_pages;
  return r;
}

// The kernels use sm_103a instructions (tcgen05-era conversions, bulk copies).
qsa_status_t check_device() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return QSA_ERR_CUDA;
  }
  int major = 0, minor = 0;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess) {
    cudaGetLastError();
    return QSA_ERR_CUDA;
  }
  if (major != 10 || minor != 3) return QSA_ERR_UNSUPPORTED;
  return QSA_OK;
}

qsa_status_t from_cuda(cudaError_t e) {
  if (e == cudaSuccess) e = cudaGetLastError();
  else cudaGetLastError();
  return e == cudaSuccess ? QSA_OK : QSA_ERR_CUDA;
}

qsa_status_t check_decode_args(const qsa_geom_t* geom, int k) {
  qsa_status_t st = check_geom(geom);
  if (st != QSA_OK) return st;
  if (k < 1) return QSA_ERR_INVALID_ARG;
  if (k > qsa::kMaxK) return QSA_ERR_UNSUPPORTED;
  if ((long long)geom->rows_per_req * k > qsa::kMaxUnion) return QSA_ERR_UNSUPPORTED;
  return QSA_OK;
}

// A row of `heads` heads of D elements, 16-byte pieces.
bool rows_ok(const void* p, int64_t stride, int heads, int d) {
  return p && aligned(p, 16) && stride >= (int64_t)heads * d && stride % 8 == 0 &&
         stride < (1LL << 40);
}

// What qsa_qk_norm_rope and qsa_store_kv_tokens_rope check alike.
qsa_status_t check_norm_rope(const qsa_geom_t* geom, const qsa_norm_rope_t* nr, const void* q,
                             int64_t q_stride, const void* k, int64_t k_stride,
                             const void* q_weight, const void* k_weight, const float* cs,
                             const void* q_out) {
  qsa_status_t st = check_geom(geom, qsa::kMaxContextRows);
  if (st != QSA_OK) return st;
  if (!nr || nr->rotary_dim < 0 || nr->rotary_dim > geom->head_dim || nr->rotary_dim % 16 != 0)
    return QSA_ERR_INVALID_ARG;
  if (!(nr->eps >= 0.f) || !isfinite(nr->eps)) return QSA_ERR_INVALID_ARG;
  if ((q == nullptr) != (q_out == nullptr)) return QSA_ERR_INVALID_ARG;
  if (q && !rows_ok(q, q_stride, geom->num_q_heads, geom->head_dim)) return QSA_ERR_INVALID_ARG;
  if (!rows_ok(k, k_stride, geom->num_kv_heads, geom->head_dim)) return QSA_ERR_INVALID_ARG;
  if (!aligned(q_out, 16) || !aligned(q_weight, 16) || !aligned(k_weight, 16) || !aligned(cs, 16))
    return QSA_ERR_INVALID_ARG;
  if (nr->rotary_dim > 0 && !cs) return QSA_ERR_INVALID_ARG;
  // in place only where every row is read and written at the same address
  if (q && q_out == q && q_stride != (int64_t)geom->num_q_heads * geom->head_dim)
    return QSA_ERR_INVALID_ARG;
  return QSA_OK;
}

qsa::NormRope to_norm_rope(const qsa_norm_rope_t* nr) {
  qsa::NormRope r;
  r.rot = nr->rotary_dim;
  r.interleaved = nr->interleaved != 0;
  r.plus_one = nr->weight_plus_one != 0;
  r.eps = nr->eps;
  return r;
}

// What the calls on the 8-bit cache's rows check alike, and their common arguments.
qsa_status_t cache8_args(const qsa_geom_t* geom, const int32_t* cu_rows, int64_t total_rows,
                         const int32_t* page_table, const int32_t* seqlens, const uint8_t* k_pool,
                         const uint8_t* k_exp, const uint8_t* v_pool, const uint8_t* v_exp,
                         qsa::Cache8Args* a) {
  const qsa_status_t st = check_geom(geom, qsa::kMaxContextRows);
  if (st != QSA_OK) return st;
  if (!page_table || !seqlens || !k_pool || !k_exp || !v_pool || !v_exp) return QSA_ERR_INVALID_ARG;
  if (!aligned(k_pool, 16) || !aligned(v_pool, 16)) return QSA_ERR_INVALID_ARG;
  if (cu_rows && (total_rows < 0 || total_rows > kMaxPackedRows)) return QSA_ERR_INVALID_ARG;
  a->cu = cu_rows;
  a->rows = cu_rows ? total_rows : (int64_t)geom->batch * geom->rows_per_req;
  a->page_table = page_table;
  a->seqlens = seqlens;
  a->k_pool = const_cast<uint8_t*>(k_pool);   // (the read-back only reads them)
  a->k_exp = const_cast<uint8_t*>(k_exp);
  a->v_pool = const_cast<uint8_t*>(v_pool);
  a->v_exp = const_cast<uint8_t*>(v_exp);
  return QSA_OK;
}

qsa_status_t check_dense_geom(const qsa_geom_t* geom) {
  qsa_status_t st = check_geom(geom, qsa::kMaxContextRows);
  if (st != QSA_OK) return st;
  return geom->num_q_heads / geom->num_kv_heads > 128 ? QSA_ERR_UNSUPPORTED : QSA_OK;
}

qsa_status_t check_prompt(const qsa_geom_t* geom, int64_t total_rows) {
  const qsa_status_t st = check_dense_geom(geom);
  if (st != QSA_OK) return st;
  return total_rows < 0 || total_rows > kMaxPackedRows ? QSA_ERR_INVALID_ARG : QSA_OK;
}

}  // namespace

namespace qsa {
unsigned long long wait_limit_ns() { return g_wait_ns.load(std::memory_order_relaxed); }
}  // namespace qsa

extern "C" {

void qsa_debug_set_wait_ns(unsigned long long ns) {
  g_wait_ns.store(ns == 0 ? kDefaultWaitNs : ns, std::memory_order_relaxed);
}

int qsa_debug_bounds_status(void) {
#ifdef QSA_DEBUG_BOUNDS
  if (cudaDeviceSynchronize() != cudaSuccess) {
    cudaGetLastError();
    return -1;
  }
  int first = 0;
  for (int v : {qsa::bounds_word_attend(), qsa::bounds_word_decode(), qsa::bounds_word_index(),
                qsa::bounds_word_select(), qsa::bounds_word_store(), qsa::bounds_word_rollback(),
                qsa::bounds_word_prefill(), qsa::bounds_word_prologue(), qsa::bounds_word_dense(),
                qsa::bounds_word_dense_tile(), qsa::bounds_word_cache8(),
                qsa::bounds_word_dense8(), qsa::bounds_word_prompt()}) {
    if (v < 0) return -1;
    if (first == 0) first = v;
  }
  return first;
#else
  return -1;
#endif
}

const char* qsa_status_string(qsa_status_t s) {
  switch (s) {
    case QSA_OK: return "ok";
    case QSA_ERR_INVALID_ARG: return "invalid argument";
    case QSA_ERR_UNSUPPORTED: return "unsupported shape or device (needs sm_103)";
    case QSA_ERR_CUDA: return "CUDA error";
    case QSA_ERR_WORKSPACE: return "workspace missing or too small";
    case QSA_ERR_DEVICE_TIMEOUT: return "a bounded device-side wait timed out";
  }
  return "unknown status";
}

qsa_status_t qsa_store_kv_tokens(const qsa_geom_t* geom, const void* k_new_bf16,
                                 const void* v_new_bf16, const int8_t* ik_new, float k_scale,
                                 float v_scale, const int32_t* page_table,
                                 const int32_t* seqlens, uint8_t* k_pool, uint8_t* k_sf,
                                 uint8_t* v_pool, uint8_t* v_sf, int8_t* ik_pool,
                                 cudaStream_t stream) {
  qsa_status_t st = check_geom(geom, qsa::kMaxContextRows);
  if (st != QSA_OK) return st;
  if (!k_new_bf16 || !v_new_bf16 || !ik_new || !page_table || !seqlens || !k_pool || !k_sf ||
      !v_pool || !v_sf || !ik_pool)
    return QSA_ERR_INVALID_ARG;
  if (!(k_scale > 0.f) || !(v_scale > 0.f) || !isfinite(k_scale) || !isfinite(v_scale))
    return QSA_ERR_INVALID_ARG;
  // A lane moves D/32 values: 8 or 16 bytes of bf16 in, 2 or 4 code bytes out.
  const uintptr_t in_al = geom->head_dim / 16, out_al = geom->head_dim / 64;
  if (!aligned(k_new_bf16, in_al) || !aligned(v_new_bf16, in_al) || !aligned(ik_new, 4) ||
      !aligned(ik_pool, 4) || !aligned(k_pool, out_al) || !aligned(v_pool, out_al))
    return QSA_ERR_INVALID_ARG;
  st = check_device();
  if (st != QSA_OK) return st;
  return from_cuda(qsa::launch_store_tokens(to_geom(geom), k_new_bf16, v_new_bf16, ik_new,
                                            k_scale, v_scale, page_table, seqlens, k_pool, k_sf,
                                            v_pool, v_sf, ik_pool, true, stream));
}

size_t qsa_rollback_state_bytes(const qsa_geom_t* geom) {
  if (check_geom(geom) != QSA_OK) return 0;
  return (size_t)geom->batch * geom->rows_per_req * qsa::rollback_row_bytes(geom->num_kv_heads, geom->head_dim);
}

qsa_status_t qsa_rollback_gather(const qsa_geom_t* geom, const int32_t* page_table,
                                 const int32_t* seqlens, const uint8_t* k_pool,
                                 const uint8_t* k_sf, const uint8_t* v_pool, const uint8_t* v_sf,
                                 const int8_t* ik_pool, void* saved, cudaStream_t stream) {
  qsa_status_t st = check_geom(geom);
  if (st != QSA_OK) return st;
  if (!page_table || !seqlens || !k_pool || !k_sf || !v_pool || !v_sf || !ik_pool || !saved)
    return QSA_ERR_INVALID_ARG;
  if (!aligned(k_pool, 4) || !aligned(k_sf, 4) || !aligned(v_pool, 4) || !aligned(v_sf, 4) ||
      !aligned(ik_pool, 4) || !aligned(saved, 4))
    return QSA_ERR_INVALID_ARG;
  st = check_device();
  if (st != QSA_OK) return st;
  return from_cuda(qsa::launch_rollback(
      to_geom(geom), false, page_table, seqlens, nullptr, const_cast<uint8_t*>(k_pool),
      const_cast<uint8_t*>(k_sf), const_cast<uint8_t*>(v_pool), const_cast<uint8_t*>(v_sf),
      const_cast<int8_t*>(ik_pool), reinterpret_cast<uint8_t*>(saved), true, stream));
}

qsa_status_t qsa_rollback_restore(const qsa_geom_t* geom, const int32_t* page_table,
                                  const int32_t* seqlens, const int32_t* rejected,
                                  const void* saved, uint8_t* k_pool, uint8_t* k_sf,
                                  uint8_t* v_pool, uint8_t* v_sf, int8_t* ik_pool,
                                  cudaStream_t stream) {
  qsa_status_t st = check_geom(geom);
  if (st != QSA_OK) return st;
  if (!page_table || !seqlens || !rejected || !saved || !k_pool || !k_sf || !v_pool || !v_sf ||
      !ik_pool)
    return QSA_ERR_INVALID_ARG;
  if (!aligned(k_pool, 4) || !aligned(k_sf, 4) || !aligned(v_pool, 4) || !aligned(v_sf, 4) ||
      !aligned(ik_pool, 4) || !aligned(saved, 4))
    return QSA_ERR_INVALID_ARG;
  st = check_device();
  if (st != QSA_OK) return st;
  return from_cuda(qsa::launch_rollback(to_geom(geom), true, page_table, seqlens, rejected,
                                        k_pool, k_sf, v_pool, v_sf, ik_pool,
                                        const_cast<uint8_t*>(reinterpret_cast<const uint8_t*>(saved)),
                                        true, stream));
}

qsa_status_t qsa_index_scores(const qsa_geom_t* geom, const int8_t* iq, const int8_t* ik_pool,
                              const int32_t* page_table, const int32_t* seqlens,
                              int32_t* scores, cudaStream_t stream) {
  qsa_status_t st = check_geom(geom, qsa::kMaxContextRows);
  if (st != QSA_OK) return st;
  if (!iq || !ik_pool || !page_table || !seqlens || !scores) return QSA_ERR_INVALID_ARG;
  if (!aligned(ik_pool, 16) || !aligned(iq, 16)) return QSA_ERR_INVALID_ARG;
  st = check_device();
  if (st != QSA_OK) return st;
  return from_cuda(qsa::launch_index_scores(to_geom(geom), iq, ik_pool, page_table, seqlens,
                                            scores, true, stream));
}

qsa_status_t qsa_select_topk(const qsa_geom_t* geom, const int32_t* scores,
                             const int32_t* seqlens, int k, int window, int32_t* sel,
                             int32_t* nsel, cudaStream_t stream) {
  qsa_status_t st = check_geom(geom, qsa::kMaxContextRows);
  if (st != QSA_OK) return st;
  if (!scores || !seqlens || !sel || !nsel) return QSA_ERR_INVALID_ARG;
  if (k < 1 || window < 0 || window > k) return QSA_ERR_INVALID_ARG;
  if (k > qsa::kMaxK) return QSA_ERR_UNSUPPORTED;
  st = check_device();
  if (st != QSA_OK) return st;
  return from_cuda(qsa::launch_select_topk(to_geom(geom), scores, seqlens, k, window, sel, nsel,
                                           true, stream));
}

size_t qsa_sparse_decode_workspace_bytes_ex(const qsa_geom_t* geom, int k, int num_splits) {
  if (check_decode_args(geom, k) != QSA_OK || num_splits < 0) return 0;
  return qsa::plan_sparse_decode(to_geom(geom), k, num_splits).ws_bytes;
}

size_t qsa_sparse_decode_workspace_bytes(const qsa_geom_t* geom, int k) {
  return qsa_sparse_decode_workspace_bytes_ex(geom, k, 0);
}

qsa_status_t qsa_workspace_init(void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (!workspace || workspace_bytes == 0) return QSA_ERR_INVALID_ARG;
  return from_cuda(cudaMemsetAsync(workspace, 0, workspace_bytes, stream));
}

qsa_status_t qsa_sparse_decode_ex(const qsa_geom_t* geom, const void* q_bf16,
                                  const uint8_t* k_pool, const uint8_t* k_sf,
                                  const uint8_t* v_pool, const uint8_t* v_sf, float k_scale,
                                  float v_scale, float sm_scale, const int32_t* page_table,
                                  const int32_t* seqlens, const int32_t* sel, int k,
                                  void* out_bf16, float* lse, void* workspace,
                                  size_t workspace_bytes, int num_splits, cudaStream_t stream) {
  qsa_status_t st = check_decode_args(geom, k);
  if (st != QSA_OK) return st;
  if (num_splits < 0) return QSA_ERR_INVALID_ARG;
  if (!q_bf16 || !k_pool || !k_sf || !v_pool || !v_sf || !page_table || !seqlens || !sel ||
      !out_bf16 || !lse)
    return QSA_ERR_INVALID_ARG;
  if (!aligned(k_pool, 16) || !aligned(v_pool, 16) || !aligned(k_sf, 16) || !aligned(v_sf, 16) ||
      !aligned(q_bf16, 8))
    return QSA_ERR_INVALID_ARG;
  const Geom g = to_geom(geom);
  const qsa::DecodePlan plan = qsa::plan_sparse_decode(g, k, num_splits);
  if (!workspace || workspace_bytes < plan.ws_bytes || !aligned(workspace, 256))
    return QSA_ERR_WORKSPACE;
  st = check_device();
  if (st != QSA_OK) return st;
  // Verify rows launch without programmatic dependent launch: their grid is
  // planned to fill every CTA slot of the GPU in one wave, and CTAs placed
  // early (while the selection kernel still holds its SMs) left clusters
  // for a second wave (wide aggregated verify: 139.5 us per step with it,
  // 102.8 us without).  Decode rows keep the overlap.
  return from_cuda(qsa::launch_sparse_decode(g, plan, q_bf16, k_pool, k_sf, v_pool, v_sf, k_scale,
                                             v_scale, sm_scale, page_table, seqlens, sel, k,
                                             out_bf16, lse, workspace, g.R == 1, stream));
}

// Context row groups: head_dim 128 or 256, a head group of at most 128 heads,
// and a tile's selections + union within the CTA's shared memory.
qsa_status_t check_prefill_args(const qsa_geom_t* geom, int k) {
  qsa_status_t st = check_geom(geom, qsa::kMaxContextRows);
  if (st != QSA_OK) return st;
  if (k < 1) return QSA_ERR_INVALID_ARG;
  if (k > qsa::kMaxK || (geom->head_dim != 128 && geom->head_dim != 256))
    return QSA_ERR_UNSUPPORTED;
  const Geom g = to_geom(geom);
  if (qsa::prefill_rows_per_tile(g) < 1) return QSA_ERR_UNSUPPORTED;
  if (qsa::prefill_smem_bytes(g, k) > 227 * 1024) return QSA_ERR_UNSUPPORTED;
  return QSA_OK;
}

size_t qsa_sparse_prefill_workspace_bytes(const qsa_geom_t* geom, int k) {
  return check_prefill_args(geom, k) == QSA_OK ? 256 : 0;
}

qsa_status_t qsa_sparse_prefill(const qsa_geom_t* geom, const void* q_bf16,
                                const uint8_t* k_pool, const uint8_t* k_sf,
                                const uint8_t* v_pool, const uint8_t* v_sf, float k_scale,
                                float v_scale, float sm_scale, const int32_t* page_table,
                                const int32_t* seqlens, const int32_t* sel, int k,
                                void* out_bf16, float* lse, void* workspace,
                                size_t workspace_bytes, cudaStream_t stream) {
  qsa_status_t st = check_prefill_args(geom, k);
  if (st != QSA_OK) return st;
  if (!q_bf16 || !k_pool || !k_sf || !v_pool || !v_sf || !page_table || !seqlens || !sel ||
      !out_bf16 || !lse)
    return QSA_ERR_INVALID_ARG;
  if (!aligned(k_pool, 16) || !aligned(v_pool, 16) || !aligned(k_sf, 16) || !aligned(v_sf, 16) ||
      !aligned(q_bf16, 16) || !aligned(out_bf16, 16))
    return QSA_ERR_INVALID_ARG;
  if (!(k_scale > 0.f) || !(sm_scale > 0.f) || !isfinite(k_scale) || !isfinite(sm_scale) ||
      !isfinite(v_scale))
    return QSA_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < 256 || !aligned(workspace, 256)) return QSA_ERR_WORKSPACE;
  st = check_device();
  if (st != QSA_OK) return st;
  return from_cuda(qsa::launch_sparse_prefill(to_geom(geom), q_bf16, k_pool, k_sf, v_pool, v_sf,
                                              k_scale, v_scale, sm_scale, page_table, seqlens,
                                              sel, k, out_bf16, lse,
                                              reinterpret_cast<int*>(workspace), stream));
}

qsa_status_t qsa_rope_init(const qsa_rope_config_t* config, qsa_rope_t* rope) {
  if (!rope) return QSA_ERR_INVALID_ARG;
  qsa_status_t st = check_rope_config(config);
  if (st != QSA_OK) return st;
  qsa_rope_t plan = {};
  st = spectrum(*config, config->rotary_dim / 2, plan.turns);
  if (st == QSA_OK) st = finish_plan(*config, &plan);
  if (st == QSA_OK) *rope = plan;
  return st;
}

qsa_status_t qsa_rope_axes_init(const qsa_rope_config_t* config, int axes, const int* pairs,
                                int layout, qsa_rope_axes_t* plan) {
  if (!pairs || !plan) return QSA_ERR_INVALID_ARG;
  qsa_status_t st = check_rope_config(config);
  if (st != QSA_OK) return st;
  if (axes < 1 || axes > QSA_ROPE_MAX_AXES) return QSA_ERR_INVALID_ARG;
  if (layout < QSA_AXES_SECTIONS || layout > QSA_AXES_SPECTRA) return QSA_ERR_INVALID_ARG;
  const int all = config->rotary_dim / 2;
  int left = all;
  for (int a = 0; a < axes; ++a) {
    if (pairs[a] < 1 || pairs[a] > left) return QSA_ERR_INVALID_ARG;
    left -= pairs[a];
  }
  if (left != 0) return QSA_ERR_INVALID_ARG;
  qsa_rope_axes_t p = {};
  p.axes = axes;
  if (layout == QSA_AXES_INTERLEAVED) {
    int count[QSA_ROPE_MAX_AXES] = {};
    for (int i = 0; i < all; ++i) {
      const int a = i % axes;
      p.axis[i] = (uint8_t)(a > 0 && i < axes * pairs[a] ? a : 0);
      ++count[p.axis[i]];
    }
    for (int a = 0; a < axes; ++a)
      if (count[a] != pairs[a]) return QSA_ERR_INVALID_ARG;
  } else {
    for (int a = 0, i = 0; a < axes; ++a)
      for (int j = 0; j < pairs[a]; ++j) p.axis[i++] = (uint8_t)a;
  }
  if (layout == QSA_AXES_SPECTRA) {
    for (int a = 0, i = 0; a < axes && st == QSA_OK; i += pairs[a++])
      st = spectrum(*config, pairs[a], p.rope.turns + i);
  } else {
    st = spectrum(*config, all, p.rope.turns);
  }
  if (st == QSA_OK) st = finish_plan(*config, &p.rope);
  if (st == QSA_OK) *plan = p;
  return st;
}

qsa_status_t qsa_rope_axes_rows(const qsa_rope_axes_t* plan, const int32_t* positions,
                                int64_t rows, float* cs, cudaStream_t stream) {
  if (!plan || !positions || !cs || !aligned(cs, 16)) return QSA_ERR_INVALID_ARG;
  if (!plan_ok(plan->rope) || plan->axes < 1 || plan->axes > QSA_ROPE_MAX_AXES)
    return QSA_ERR_INVALID_ARG;
  for (int i = 0; i < plan->rope.rotary_dim / 2; ++i)
    if (plan->axis[i] >= plan->axes) return QSA_ERR_INVALID_ARG;
  if (rows < 0 || rows > kMaxPackedRows) return QSA_ERR_INVALID_ARG;
  const qsa_status_t st = check_device();
  if (st != QSA_OK || rows == 0) return st;
  return from_cuda(qsa::launch_rope_axes(*plan, positions, rows, cs, true, stream));
}

qsa_status_t qsa_rope_rows(const qsa_geom_t* geom, const qsa_rope_t* rope, const int32_t* seqlens,
                           const int32_t* positions, float* cs, cudaStream_t stream) {
  qsa_status_t st = check_geom(geom, qsa::kMaxContextRows);
  if (st != QSA_OK) return st;
  if (!rope || (!seqlens && !positions) || !cs || !aligned(cs, 8)) return QSA_ERR_INVALID_ARG;
  if (!plan_ok(*rope)) return QSA_ERR_INVALID_ARG;
  st = check_device();
  if (st != QSA_OK) return st;
  return from_cuda(qsa::launch_rope_rows(to_geom(geom), *rope, seqlens, positions, cs, true, stream));
}

qsa_status_t qsa_qk_norm_rope(const qsa_geom_t* geom, const qsa_norm_rope_t* norm_rope,
                              const void* q_bf16, int64_t q_row_stride, const void* k_bf16,
                              int64_t k_row_stride, const void* q_weight_bf16,
                              const void* k_weight_bf16, const float* cs, void* q_out_bf16,
                              void* k_out_bf16, cudaStream_t stream) {
  qsa_status_t st = check_norm_rope(geom, norm_rope, q_bf16, q_row_stride, k_bf16, k_row_stride,
                                    q_weight_bf16, k_weight_bf16, cs, q_out_bf16);
  if (st != QSA_OK) return st;
  if (!k_out_bf16 || !aligned(k_out_bf16, 16)) return QSA_ERR_INVALID_ARG;
  if (k_out_bf16 == k_bf16 && k_row_stride != (int64_t)geom->num_kv_heads * geom->head_dim)
    return QSA_ERR_INVALID_ARG;
  st = check_device();
  if (st != QSA_OK) return st;
  qsa::PrologueArgs a = {};
  a.q = reinterpret_cast<const __nv_bfloat16*>(q_bf16);
  a.k = reinterpret_cast<const __nv_bfloat16*>(k_bf16);
  a.q_stride = q_row_stride;
  a.k_stride = k_row_stride;
  a.q_weight = reinterpret_cast<const __nv_bfloat16*>(q_weight_bf16);
  a.k_weight = reinterpret_cast<const __nv_bfloat16*>(k_weight_bf16);
  a.cs = cs;
  a.q_out = reinterpret_cast<__nv_bfloat16*>(q_out_bf16);
  a.k_out = reinterpret_cast<__nv_bfloat16*>(k_out_bf16);
  return from_cuda(qsa::launch_prologue(to_geom(geom), to_norm_rope(norm_rope), a, true, stream));
}

qsa_status_t qsa_store_kv_tokens_rope(const qsa_geom_t* geom, const qsa_norm_rope_t* norm_rope,
                                      const void* q_bf16, int64_t q_row_stride,
                                      const void* k_bf16, int64_t k_row_stride,
                                      const void* v_bf16, int64_t v_row_stride,
                                      const int8_t* ik_new, const void* q_weight_bf16,
                                      const void* k_weight_bf16, const float* cs, float k_scale,
                                      float v_scale, const int32_t* page_table,
                                      const int32_t* seqlens, void* q_out_bf16, uint8_t* k_pool,
                                      uint8_t* k_sf, uint8_t* v_pool, uint8_t* v_sf,
                                      int8_t* ik_pool, cudaStream_t stream) {
  qsa_status_t st = check_norm_rope(geom, norm_rope, q_bf16, q_row_stride, k_bf16, k_row_stride,
                                    q_weight_bf16, k_weight_bf16, cs, q_out_bf16);
  if (st != QSA_OK) return st;
  if (!rows_ok(v_bf16, v_row_stride, geom->num_kv_heads, geom->head_dim)) return QSA_ERR_INVALID_ARG;
  if (!ik_new || !page_table || !seqlens || !k_pool || !k_sf || !v_pool || !v_sf || !ik_pool)
    return QSA_ERR_INVALID_ARG;
  if (!positive(k_scale) || !positive(v_scale)) return QSA_ERR_INVALID_ARG;
  if (!aligned(ik_new, 4) || !aligned(ik_pool, 4) || !aligned(k_pool, 4) || !aligned(v_pool, 4))
    return QSA_ERR_INVALID_ARG;
  st = check_device();
  if (st != QSA_OK) return st;
  qsa::PrologueArgs a = {};
  a.q = reinterpret_cast<const __nv_bfloat16*>(q_bf16);
  a.k = reinterpret_cast<const __nv_bfloat16*>(k_bf16);
  a.v = reinterpret_cast<const __nv_bfloat16*>(v_bf16);
  a.q_stride = q_row_stride;
  a.k_stride = k_row_stride;
  a.v_stride = v_row_stride;
  a.ik = ik_new;
  a.q_weight = reinterpret_cast<const __nv_bfloat16*>(q_weight_bf16);
  a.k_weight = reinterpret_cast<const __nv_bfloat16*>(k_weight_bf16);
  a.cs = cs;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.page_table = page_table;
  a.seqlens = seqlens;
  a.q_out = reinterpret_cast<__nv_bfloat16*>(q_out_bf16);
  a.k_pool = k_pool;
  a.k_sf = k_sf;
  a.v_pool = v_pool;
  a.v_sf = v_sf;
  a.ik_pool = ik_pool;
  return from_cuda(qsa::launch_prologue(to_geom(geom), to_norm_rope(norm_rope), a, true, stream));
}

qsa_status_t qsa_load_kv_tokens(const qsa_geom_t* geom, const int32_t* page_table,
                                const int32_t* seqlens, const uint8_t* k_pool,
                                const uint8_t* k_sf, const uint8_t* v_pool, const uint8_t* v_sf,
                                float k_scale, float v_scale, void* k_out_bf16,
                                void* v_out_bf16, cudaStream_t stream) {
  qsa_status_t st = check_geom(geom, qsa::kMaxContextRows);
  if (st != QSA_OK) return st;
  if (!page_table || !seqlens || !k_pool || !k_sf || !v_pool || !v_sf || !k_out_bf16 || !v_out_bf16)
    return QSA_ERR_INVALID_ARG;
  if (!isfinite(k_scale) || !isfinite(v_scale)) return QSA_ERR_INVALID_ARG;
  if (!aligned(k_pool, 4) || !aligned(v_pool, 4) || !aligned(k_out_bf16, 16) ||
      !aligned(v_out_bf16, 16))
    return QSA_ERR_INVALID_ARG;
  st = check_device();
  if (st != QSA_OK) return st;
  return from_cuda(qsa::launch_load_tokens(to_geom(geom), page_table, seqlens, k_pool, k_sf, v_pool,
                                           v_sf, k_scale, v_scale, k_out_bf16, v_out_bf16, true,
                                           stream));
}

qsa_status_t qsa_store_kv_tokens_fp8(const qsa_geom_t* geom, const void* k_bf16,
                                     int64_t k_row_stride, const void* v_bf16,
                                     int64_t v_row_stride, const int32_t* cu_rows,
                                     int64_t total_rows, const int32_t* page_table,
                                     const int32_t* seqlens, uint8_t* k_pool, uint8_t* k_exp,
                                     uint8_t* v_pool, uint8_t* v_exp, cudaStream_t stream) {
  qsa::Cache8Args a = {};
  qsa_status_t st = cache8_args(geom, cu_rows, total_rows, page_table, seqlens, k_pool, k_exp,
                                v_pool, v_exp, &a);
  if (st != QSA_OK) return st;
  if (!rows_ok(k_bf16, k_row_stride, geom->num_kv_heads, geom->head_dim) ||
      !rows_ok(v_bf16, v_row_stride, geom->num_kv_heads, geom->head_dim))
    return QSA_ERR_INVALID_ARG;
  st = check_device();
  if (st != QSA_OK || a.rows == 0) return st;
  a.k = reinterpret_cast<const __nv_bfloat16*>(k_bf16);
  a.v = reinterpret_cast<const __nv_bfloat16*>(v_bf16);
  a.k_stride = k_row_stride;
  a.v_stride = v_row_stride;
  return from_cuda(qsa::launch_cache8(to_geom(geom), a, true, true, stream));
}

qsa_status_t qsa_load_kv_tokens_fp8(const qsa_geom_t* geom, const int32_t* cu_rows,
                                    int64_t total_rows, const int32_t* page_table,
                                    const int32_t* seqlens, const uint8_t* k_pool,
                                    const uint8_t* k_exp, const uint8_t* v_pool,
                                    const uint8_t* v_exp, void* k_out_bf16, void* v_out_bf16,
                                    cudaStream_t stream) {
  qsa::Cache8Args a = {};
  qsa_status_t st = cache8_args(geom, cu_rows, total_rows, page_table, seqlens, k_pool, k_exp,
                                v_pool, v_exp, &a);
  if (st != QSA_OK) return st;
  if (!k_out_bf16 || !v_out_bf16 || !aligned(k_out_bf16, 16) || !aligned(v_out_bf16, 16))
    return QSA_ERR_INVALID_ARG;
  st = check_device();
  if (st != QSA_OK || a.rows == 0) return st;
  a.k_out = reinterpret_cast<__nv_bfloat16*>(k_out_bf16);
  a.v_out = reinterpret_cast<__nv_bfloat16*>(v_out_bf16);
  return from_cuda(qsa::launch_cache8(to_geom(geom), a, false, true, stream));
}

size_t qsa_dense_attention_workspace_bytes(const qsa_geom_t* geom) {
  return check_dense_geom(geom) == QSA_OK ? qsa::dense_workspace_bytes(to_geom(geom)) : 0;
}

qsa_status_t qsa_dense_attention(const qsa_geom_t* geom, const void* q_bf16,
                                 const uint8_t* k_pool, const uint8_t* k_sf,
                                 const uint8_t* v_pool, const uint8_t* v_sf, float k_scale,
                                 float v_scale, float sm_scale, const int32_t* page_table,
                                 const int32_t* seqlens, int window, const float* sinks,
                                 void* out_bf16, float* lse, void* workspace,
                                 size_t workspace_bytes, cudaStream_t stream) {
  qsa_status_t st = check_dense_geom(geom);
  if (st != QSA_OK) return st;
  if (!q_bf16 || !k_pool || !k_sf || !v_pool || !v_sf || !page_table || !seqlens || !out_bf16 || !lse)
    return QSA_ERR_INVALID_ARG;
  if (window < 0) return QSA_ERR_INVALID_ARG;
  if (!aligned(k_pool, 16) || !aligned(v_pool, 16) || !aligned(k_sf, 16) || !aligned(v_sf, 16) ||
      !aligned(q_bf16, 16) || !aligned(out_bf16, 16))
    return QSA_ERR_INVALID_ARG;
  if (!positive(k_scale) || !positive(sm_scale) || !isfinite(v_scale)) return QSA_ERR_INVALID_ARG;
  const Geom g = to_geom(geom);
  if (!workspace || workspace_bytes < qsa::dense_workspace_bytes(g) || !aligned(workspace, 256))
    return QSA_ERR_WORKSPACE;
  st = check_device();
  if (st != QSA_OK) return st;
  qsa::DenseArgs a = {};
  a.q = q_bf16;
  a.k_pool = k_pool; a.k_sf = k_sf; a.v_pool = v_pool; a.v_sf = v_sf;
  a.k_scale = k_scale; a.v_scale = v_scale; a.sm_scale = sm_scale;
  a.page_table = page_table; a.seqlens = seqlens;
  a.window = window; a.sinks = sinks;
  a.out = out_bf16; a.lse = lse; a.workspace = workspace;
  return from_cuda(qsa::launch_dense(g, a, stream));
}

size_t qsa_dense_attention_fp8_workspace_bytes(const qsa_geom_t* geom) {
  return check_dense_geom(geom) == QSA_OK ? qsa::dense8_workspace_bytes(to_geom(geom)) : 0;
}

qsa_status_t qsa_dense_attention_fp8(const qsa_geom_t* geom, const void* q_bf16,
                                     const uint8_t* k_pool, const uint8_t* k_exp,
                                     const uint8_t* v_pool, const uint8_t* v_exp, float sm_scale,
                                     const int32_t* page_table, const int32_t* seqlens, int window,
                                     const float* sinks, void* out_bf16, float* lse,
                                     void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  qsa_status_t st = check_dense_geom(geom);
  if (st != QSA_OK) return st;
  if (!q_bf16 || !k_pool || !k_exp || !v_pool || !v_exp || !page_table || !seqlens || !out_bf16 || !lse)
    return QSA_ERR_INVALID_ARG;
  if (window < 0) return QSA_ERR_INVALID_ARG;
  if (!aligned(k_pool, 16) || !aligned(v_pool, 16) || !aligned(k_exp, 16) || !aligned(v_exp, 16) ||
      !aligned(q_bf16, 16) || !aligned(out_bf16, 16))
    return QSA_ERR_INVALID_ARG;
  if (!positive(sm_scale)) return QSA_ERR_INVALID_ARG;
  const Geom g = to_geom(geom);
  if (!workspace || workspace_bytes < qsa::dense8_workspace_bytes(g) || !aligned(workspace, 256))
    return QSA_ERR_WORKSPACE;
  st = check_device();
  if (st != QSA_OK) return st;
  qsa::DenseArgs a = {};
  a.q = q_bf16;
  a.k_pool = k_pool; a.k_sf = k_exp; a.v_pool = v_pool; a.v_sf = v_exp;
  a.sm_scale = sm_scale;
  a.page_table = page_table; a.seqlens = seqlens;
  a.window = window; a.sinks = sinks;
  a.out = out_bf16; a.lse = lse; a.workspace = workspace;
  return from_cuda(qsa::launch_dense8(g, a, stream));
}

size_t qsa_prompt_attention_workspace_bytes(const qsa_geom_t* geom, int64_t total_rows) {
  return check_prompt(geom, total_rows) == QSA_OK ? 256 : 0;
}

qsa_status_t qsa_prompt_attention(const qsa_geom_t* geom, const void* q_bf16, int64_t q_row_stride,
                                  const void* k_bf16, int64_t k_row_stride, const void* v_bf16,
                                  int64_t v_row_stride, const int32_t* cu_seqlens,
                                  int64_t total_rows, float sm_scale, int window,
                                  const float* sinks, void* out_bf16, float* lse, void* workspace,
                                  size_t workspace_bytes, cudaStream_t stream) {
  qsa_status_t st = check_prompt(geom, total_rows);
  if (st != QSA_OK) return st;
  if (!cu_seqlens || !out_bf16 || !lse || !aligned(out_bf16, 16) || window < 0 || !positive(sm_scale))
    return QSA_ERR_INVALID_ARG;
  // (a tensor map's strides have 40 bits of bytes)
  if (!rows_ok(q_bf16, q_row_stride, geom->num_q_heads, geom->head_dim) ||
      !rows_ok(k_bf16, k_row_stride, geom->num_kv_heads, geom->head_dim) ||
      !rows_ok(v_bf16, v_row_stride, geom->num_kv_heads, geom->head_dim) ||
      q_row_stride >= (1LL << 39) || k_row_stride >= (1LL << 39) || v_row_stride >= (1LL << 39))
    return QSA_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < 256 || !aligned(workspace, 256)) return QSA_ERR_WORKSPACE;
  st = check_device();
  if (st != QSA_OK || total_rows == 0) return st;
  qsa::PromptArgs a = {};
  a.q = q_bf16; a.k = k_bf16; a.v = v_bf16;
  a.q_stride = q_row_stride; a.k_stride = k_row_stride; a.v_stride = v_row_stride;
  a.rows = total_rows;
  a.cu = cu_seqlens;
  a.sm_scale = sm_scale;
  a.window = window; a.sinks = sinks;
  a.out = out_bf16; a.lse = lse; a.workspace = workspace;
  return from_cuda(qsa::launch_prompt(to_geom(geom), a, stream));
}

int qsa_select_sparse_decode_fused(const qsa_geom_t* geom) {
  if (check_geom(geom) != QSA_OK) return 0;
  return qsa::decode_can_fuse_select(to_geom(geom)) ? 1 : 0;
}

qsa_status_t qsa_select_sparse_decode(const qsa_geom_t* geom, const int32_t* scores, int window,
                                      const void* q_bf16, const uint8_t* k_pool,
                                      const uint8_t* k_sf, const uint8_t* v_pool,
                                      const uint8_t* v_sf, float k_scale, float v_scale,
                                      float sm_scale, const int32_t* page_table,
                                      const int32_t* seqlens, int k, int32_t* sel, int32_t* nsel,
                                      void* out_bf16, float* lse, void* workspace,
                                      size_t workspace_bytes, int num_splits,
                                      cudaStream_t stream) {
  qsa_status_t st = check_decode_args(geom, k);
  if (st != QSA_OK) return st;
  if (window < 0 || window > k || num_splits < 0) return QSA_ERR_INVALID_ARG;
  if (!scores || !q_bf16 || !k_pool || !k_sf || !v_pool || !v_sf || !page_table || !seqlens ||
      !sel || !nsel || !out_bf16 || !lse)
    return QSA_ERR_INVALID_ARG;
  if (!aligned(k_pool, 16) || !aligned(v_pool, 16) || !aligned(k_sf, 16) || !aligned(v_sf, 16) ||
      !aligned(q_bf16, 8))
    return QSA_ERR_INVALID_ARG;
  const Geom g = to_geom(geom);
  const qsa::DecodePlan plan = qsa::plan_sparse_decode(g, k, num_splits);
  if (!workspace || workspace_bytes < plan.ws_bytes || !aligned(workspace, 256))
    return QSA_ERR_WORKSPACE;
  st = check_device();
  if (st != QSA_OK) return st;
  if (qsa::decode_can_fuse_select(g))
    return from_cuda(qsa::launch_sparse_decode(g, plan, q_bf16, k_pool, k_sf, v_pool, v_sf,
                                               k_scale, v_scale, sm_scale, page_table, seqlens,
                                               nullptr, k, out_bf16, lse, workspace, true, stream,
                                               scores, window, sel, nsel));
  cudaError_t e = qsa::launch_select_topk(g, scores, seqlens, k, window, sel, nsel, true, stream);
  if (e != cudaSuccess) return from_cuda(e);
  // Verify rows launch without programmatic dependent launch: their grid is
  // planned to fill every CTA slot of the GPU in one wave, and CTAs placed
  // early (while the selection kernel still holds its SMs) left clusters
  // for a second wave (wide aggregated verify: 139.5 us per step with it,
  // 102.8 us without).  Decode rows keep the overlap.
  return from_cuda(qsa::launch_sparse_decode(g, plan, q_bf16, k_pool, k_sf, v_pool, v_sf, k_scale,
                                             v_scale, sm_scale, page_table, seqlens, sel, k,
                                             out_bf16, lse, workspace, g.R == 1, stream));
}

qsa_status_t qsa_sparse_decode(const qsa_geom_t* geom, const void* q_bf16, const uint8_t* k_pool,
                               const uint8_t* k_sf, const uint8_t* v_pool, const uint8_t* v_sf,
                               float k_scale, float v_scale, float sm_scale,
                               const int32_t* page_table, const int32_t* seqlens,
                               const int32_t* sel, int k, void* out_bf16, float* lse,
                               void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  return qsa_sparse_decode_ex(geom, q_bf16, k_pool, k_sf, v_pool, v_sf, k_scale, v_scale,
                              sm_scale, page_table, seqlens, sel, k, out_bf16, lse, workspace,
                              workspace_bytes, 0, stream);
}

qsa_status_t qsa_workspace_status(const void* workspace, int* device_code, cudaStream_t stream) {
  if (!workspace || !device_code) return QSA_ERR_INVALID_ARG;
  int v = 0;
  cudaError_t e = cudaMemcpyAsync(&v, workspace, sizeof(int), cudaMemcpyDeviceToHost, stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return QSA_ERR_CUDA;
  }
  *device_code = v;
  return v == 0 ? QSA_OK : QSA_ERR_DEVICE_TIMEOUT;
}

}  // extern "C"
