// C ABI of the paged cache, the rotary and the windowed attention (include/kivi.h): argument checks and
// launches.  Host code only; the computation runs in tables.cu, rotary.cu, append.cu and attend.cu.
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "kivi.h"
#include "paged.h"

namespace {

constexpr int kHeadDim = 128;
using kivi::kMaxPagedSeqs;
constexpr int kMaxGqa = 64;
constexpr int kMaxTurnPairs = kHeadDim / 2;

bool aligned(const void* p, uintptr_t to) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
bool aligned16(const void* p) { return aligned(p, 16); }
bool status_ok(const int32_t* s) { return s == nullptr || aligned(s, 4); }
int log2i(int x) { return __builtin_ctz(static_cast<unsigned>(x)); }
bool finite(float x) { return x == x && x <= 3.0e38f && x >= -3.0e38f; }

int check_paged(const kivi_paged_config* c) {
  if (c == nullptr) return KIVI_ERR_INVALID_ARG;
  kivi_config one{};  // the rules of a cache of one block
  one.batch = 1;
  one.num_kv_heads = c->num_kv_heads;
  one.head_dim = c->head_dim;
  one.bits = c->bits;
  one.group_k = c->group_k;
  one.group_v = c->group_v;
  one.residual = c->residual;
  one.capacity = c->residual;
  const int st = kivi_check_config(&one);
  if (st != KIVI_OK) return st;
  if (c->num_pages < 1 || c->num_seqs < 1 || c->max_blocks < 1) return KIVI_ERR_INVALID_ARG;
  if (c->residual > 512 || c->num_seqs > kMaxPagedSeqs) return KIVI_ERR_UNSUPPORTED;
  const long long R = c->residual;
  if (c->max_blocks * R > 0x7fffffffll || static_cast<long long>(c->num_seqs) * c->num_kv_heads * R > 0x7fffffffll ||
      static_cast<long long>(c->num_pages) * c->num_kv_heads > 0x7fffffffll)
    return KIVI_ERR_UNSUPPORTED;
  return KIVI_OK;
}

bool pool_ok(const kivi_paged_cache* p) {
  return p != nullptr && aligned16(p->k_codes) && aligned16(p->v_codes) && aligned16(p->k_scale) && aligned16(p->k_zero) &&
         aligned16(p->v_scale) && aligned16(p->v_zero) && aligned16(p->k_res) && aligned16(p->v_res);
}

// Workspace, query and mask arguments both attention calls share; fills what does not depend on the cache.
int check_attend(int heads, int num_q_heads, float scale, int window, int sinks, const uint16_t* q, const uint16_t* out,
                 const int32_t* status, kivi::AttendArgs* a) {
  if (num_q_heads < 1 || num_q_heads % heads != 0) return KIVI_ERR_INVALID_ARG;
  if (num_q_heads / heads > kMaxGqa) return KIVI_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(out) || !finite(scale) || window < 0 || sinks < 0 || !status_ok(status))
    return KIVI_ERR_INVALID_ARG;
  a->heads = heads;
  a->gqa = num_q_heads / heads;
  a->q = q;
  a->out = const_cast<uint16_t*>(out);
  a->status = const_cast<int32_t*>(status);
  a->window = window == 0 ? 0x7fffffff : window;
  a->sinks = sinks;
  a->qscale = scale * 1.4426950408889634f;
  return KIVI_OK;
}

// 8 KB units a head of at most `blocks` R-token blocks and R residual rows is cut into.
long long max_units(int bits, int residual, long long blocks) {
  return blocks * (residual / kivi::attend_unit_tokens(bits)) + residual / kivi::kAttendResTokens;
}

// Workspace of max_rows rows; 0 where the units are past the kernel's 32-bit counts.
size_t attend_bytes(int max_rows, int heads, int num_q_heads, long long units) {
  if (num_q_heads < 1 || num_q_heads % heads != 0 || num_q_heads / heads > kMaxGqa || max_rows > kMaxPagedSeqs) return 0;
  if (max_rows * units > 0x7fffffffll) return 0;
  return kivi::attend_workspace_bytes(max_rows, heads, num_q_heads / heads, units);
}

int run_attend(const kivi::AttendArgs& a, int bits, long long units, void* ws, size_t ws_bytes, void* stream) {
  const size_t need = attend_bytes(a.max_rows, a.heads, a.heads * a.gqa, units);
  if (need == 0) return KIVI_ERR_UNSUPPORTED;
  if (!aligned(ws, 256) || ws_bytes < need) return KIVI_ERR_WORKSPACE;
  return kivi::launch_attend(a, bits, ws, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KIVI_OK : KIVI_ERR_CUDA;
}

bool heads_ok(const kivi_heads* h) {
  if (h == nullptr || h->num_heads == 0) return true;
  if (h->num_heads < 0 || !aligned16(h->x_dev) || !aligned16(h->y_dev)) return false;
  if (h->weight_dev != nullptr && !aligned16(h->weight_dev)) return false;
  const int64_t strides = h->x_batch | h->x_token | h->x_head | h->y_batch | h->y_token | h->y_head;
  return (strides & 7) == 0;
}

void set_heads(kivi::RotaryHeads* to, const kivi_heads* h, int rotate) {
  *to = kivi::RotaryHeads{};
  if (h == nullptr || h->num_heads == 0) return;
  to->x = h->x_dev;
  to->y = h->y_dev;
  to->weight = h->weight_dev;
  to->heads = h->num_heads;
  to->rotate = rotate;
  to->x_batch = h->x_batch;
  to->x_token = h->x_token;
  to->x_head = h->x_head;
  to->y_batch = h->y_batch;
  to->y_token = h->y_token;
  to->y_head = h->y_head;
}

}  // namespace

extern "C" {

size_t kivi_window_workspace_bytes(const kivi_config* cfg, int32_t num_q_heads) {
  if (kivi_check_config(cfg) != KIVI_OK) return 0;
  return attend_bytes(cfg->batch, cfg->num_kv_heads, num_q_heads, max_units(cfg->bits, cfg->residual, cfg->capacity / cfg->residual));
}

int kivi_decode_attention_window(const kivi_config* cfg, const kivi_cache* cache, const uint16_t* q_dev,
                                 int32_t num_q_heads, float scale, int32_t window, int32_t sinks, uint16_t* out_dev,
                                 void* workspace_dev, size_t workspace_bytes, int32_t* dev_status, void* stream) {
  int st = kivi_check_config(cfg);
  if (st != KIVI_OK) return st;
  if (cache == nullptr) return KIVI_ERR_INVALID_ARG;
  if (cfg->online_k || cfg->fine_groups || cfg->batch > kMaxPagedSeqs) return KIVI_ERR_UNSUPPORTED;
  const int R = cfg->residual;
  if (cache->n_quant < 0 || cache->n_quant % R != 0 || cache->n_quant > cfg->capacity || cache->n_res < 0 ||
      cache->n_res > R)
    return KIVI_ERR_STATE;
  kivi::AttendArgs a{};
  if ((st = check_attend(cfg->num_kv_heads, num_q_heads, scale, window, sinks, q_dev, out_dev, dev_status, &a)) != KIVI_OK)
    return st;
  if (cache->n_quant + cache->n_res == 0) return KIVI_ERR_EMPTY;
  if (!aligned16(cache->k_res) || !aligned16(cache->v_res)) return KIVI_ERR_INVALID_ARG;
  if (cache->n_quant > 0 && !(aligned16(cache->k_codes) && aligned16(cache->v_codes) && aligned16(cache->k_scale) &&
                              aligned16(cache->k_zero) && aligned16(cache->v_scale) && aligned16(cache->v_zero)))
    return KIVI_ERR_INVALID_ARG;
  a.k_codes = cache->k_codes;
  a.v_codes = cache->v_codes;
  a.k_scale = cache->k_scale;
  a.k_zero = cache->k_zero;
  a.v_scale = cache->v_scale;
  a.v_zero = cache->v_zero;
  a.k_res = cache->k_res;
  a.v_res = cache->v_res;
  a.rows = a.max_rows = a.q_rows = cfg->batch;
  a.len = cache->n_quant + cache->n_res;
  a.quant = cache->n_quant;
  a.blocks_per_head = cfg->capacity / R;
  if (static_cast<long long>(cfg->batch) * cfg->num_kv_heads > 0x7fffffffll / (a.blocks_per_head > 0 ? a.blocks_per_head : 1))
    return KIVI_ERR_UNSUPPORTED;
  a.lg_r = log2i(R);
  a.lg_gk = log2i(cfg->group_k);
  a.lg_gv = log2i(cfg->group_v);
  return run_attend(a, cfg->bits, max_units(cfg->bits, R, a.blocks_per_head), workspace_dev, workspace_bytes, stream);
}

int kivi_rotary_init(kivi_rotary* r, int32_t rotary_dim, int32_t interleaved, double theta, int32_t scaling, double factor,
                     double low, double high, int32_t original_positions) {
  if (r == nullptr || rotary_dim < 0 || rotary_dim > kHeadDim || rotary_dim % 16 != 0 || (interleaved != 0 && interleaved != 1))
    return KIVI_ERR_INVALID_ARG;
  if (!(theta > 1.0) || !(theta < 1e30) || scaling < KIVI_ROPE_NONE || scaling > KIVI_ROPE_RAMP) return KIVI_ERR_INVALID_ARG;
  if (scaling != KIVI_ROPE_NONE && (!(factor >= 1.0) || !(factor < 1e9))) return KIVI_ERR_INVALID_ARG;
  if ((scaling == KIVI_ROPE_BANDS || scaling == KIVI_ROPE_RAMP) && (!(low > 0.0) || !(high > low) || !(high < 1e9) || original_positions < 1))
    return KIVI_ERR_INVALID_ARG;
  *r = kivi_rotary{};
  r->rotary_dim = rotary_dim;
  r->interleaved = interleaved;
  r->magnitude = 1.0f;
  const double kTurn = 6.283185307179586476925, d = rotary_dim;
  double ramp_low = 0.0, ramp_high = 1.0;
  if (scaling == KIVI_ROPE_BASE && rotary_dim > 2) theta *= std::pow(factor, d / (d - 2.0));
  if (scaling == KIVI_ROPE_RAMP) {
    // the pair index at which theta^(-2 i / d) makes that many turns over the original context
    const double at_high = d * std::log(original_positions / (high * kTurn)) / (2.0 * std::log(theta));
    const double at_low = d * std::log(original_positions / (low * kTurn)) / (2.0 * std::log(theta));
    ramp_low = std::fmax(0.0, std::floor(at_high));
    ramp_high = std::fmin(d - 1.0, std::ceil(at_low));
    r->magnitude = static_cast<float>(0.1 * std::log(factor) + 1.0);
  }
  for (int i = 0; i < rotary_dim / 2; ++i) {
    double turns = std::pow(theta, -2.0 * i / d) / kTurn;  // below 1/6 turn per position
    double keep = 1.0;                                     // share of the unscaled frequency
    if (scaling == KIVI_ROPE_LINEAR) keep = 0.0;
    if (scaling == KIVI_ROPE_BANDS) keep = std::fmin(1.0, std::fmax(0.0, (original_positions * turns - low) / (high - low)));
    if (scaling == KIVI_ROPE_RAMP)
      keep = 1.0 - std::fmin(1.0, std::fmax(0.0, (i - ramp_low) / std::fmax(ramp_high - ramp_low, 1e-3)));
    if (scaling == KIVI_ROPE_LINEAR || scaling == KIVI_ROPE_BANDS || scaling == KIVI_ROPE_RAMP)
      turns *= keep + (1.0 - keep) / factor;
    r->turns[i] = static_cast<uint64_t>(std::ldexp(turns, 64));
  }
  return KIVI_OK;
}

int kivi_rotary_apply(const kivi_rotary* rotary, int32_t dtype, int32_t batch, int32_t tokens, const int32_t* positions_dev,
                      int32_t position0, const kivi_heads* q, const kivi_heads* k, const kivi_heads* v, float eps,
                      void* stream) {
  if (rotary == nullptr || rotary->rotary_dim < 0 || rotary->rotary_dim > kHeadDim || rotary->rotary_dim % 16 != 0 ||
      (rotary->interleaved != 0 && rotary->interleaved != 1))
    return KIVI_ERR_INVALID_ARG;
  if (dtype != KIVI_DTYPE_F16 && dtype != KIVI_DTYPE_BF16) return KIVI_ERR_UNSUPPORTED;
  if (batch < 0 || tokens < 0 || !heads_ok(q) || !heads_ok(k) || !heads_ok(v) || !(eps >= 0.0f) || !finite(eps))
    return KIVI_ERR_INVALID_ARG;
  if (positions_dev != nullptr && !aligned(positions_dev, 4)) return KIVI_ERR_INVALID_ARG;
  if (positions_dev == nullptr && position0 > 0x7fffffff - tokens) return KIVI_ERR_INVALID_ARG;  // positions are int32
  if (v != nullptr && v->num_heads > 0 && v->weight_dev != nullptr) return KIVI_ERR_INVALID_ARG;
  kivi::RotaryArgs a{};
  set_heads(&a.h[0], q, 1);
  set_heads(&a.h[1], k, 1);
  set_heads(&a.h[2], v, 0);
  const long long heads = static_cast<long long>(a.h[0].heads) + a.h[1].heads + a.h[2].heads;
  if (static_cast<long long>(batch) * tokens > 0x7fffffffll || heads > (1 << 20)) return KIVI_ERR_UNSUPPORTED;
  a.heads = static_cast<int>(heads);
  a.positions = positions_dev;
  a.position0 = position0;
  a.batch = batch;
  a.tokens = tokens;
  a.rotary_dim = rotary->rotary_dim;
  a.interleaved = rotary->interleaved;
  a.magnitude = rotary->magnitude;
  a.eps = eps;
  for (int i = 0; i < kMaxTurnPairs; ++i) a.turns[i] = rotary->turns[i];
  return kivi::launch_rotary(a, dtype, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KIVI_OK : KIVI_ERR_CUDA;
}

int kivi_paged_check_config(const kivi_paged_config* cfg) { return check_paged(cfg); }

int kivi_paged_sizes(const kivi_paged_config* cfg, size_t* out) {
  const int st = check_paged(cfg);
  if (st != KIVI_OK) return st;
  if (out == nullptr) return KIVI_ERR_INVALID_ARG;
  const size_t H = cfg->num_kv_heads, R = cfg->residual, d = kHeadDim, N = cfg->num_pages, S = cfg->num_seqs;
  out[KIVI_BUF_K_CODES] = out[KIVI_BUF_V_CODES] = N * H * R * d * cfg->bits / 8;
  out[KIVI_BUF_K_SCALE] = out[KIVI_BUF_K_ZERO] = N * H * (d / cfg->group_k) * 2;
  out[KIVI_BUF_V_SCALE] = out[KIVI_BUF_V_ZERO] = N * H * (R / cfg->group_v) * 2;
  out[KIVI_BUF_K_RES] = out[KIVI_BUF_V_RES] = S * H * R * d * 2;
  out[KIVI_BUF_BLOCK_TABLE] = S * cfg->max_blocks * 4;
  out[KIVI_BUF_FREE_PAGES] = N * 4;
  out[KIVI_BUF_QUEUE] = 16;
  return KIVI_OK;
}

int kivi_paged_build_tables(const kivi_paged_config* cfg, const kivi_paged_cache* cache, int32_t num_rows,
                            const int32_t* lens_dev, const int32_t* new_tokens_dev, int32_t* lens_out_dev,
                            int64_t* queue_out_dev, const kivi_paged_plan* plan, int32_t* dev_status, void* stream) {
  const int st = check_paged(cfg);
  if (st != KIVI_OK) return st;
  if (cache == nullptr || plan == nullptr || num_rows < 0 || num_rows > cfg->num_seqs) return KIVI_ERR_INVALID_ARG;
  if (!aligned16(cache->block_table) || !aligned16(cache->free_pages) || !aligned16(cache->queue)) return KIVI_ERR_INVALID_ARG;
  if (num_rows > 0 && (!aligned(lens_dev, 4) || !aligned(new_tokens_dev, 4) || !aligned(lens_out_dev, 4)))
    return KIVI_ERR_INVALID_ARG;
  if (!aligned(queue_out_dev, 8) || !status_ok(dev_status)) return KIVI_ERR_INVALID_ARG;
  if (!aligned16(plan->cu_tokens) || !aligned16(plan->positions) || !aligned16(plan->runs) || !aligned16(plan->counts) ||
      plan->max_tokens < 1 || static_cast<long long>(plan->max_runs) < 2ll * cfg->num_seqs + plan->max_tokens / cfg->residual)
    return KIVI_ERR_INVALID_ARG;
  kivi::TablesArgs a{};
  a.lens = lens_dev;
  a.new_tokens = new_tokens_dev;
  a.lens_out = lens_out_dev;
  a.block_table = cache->block_table;
  a.free_pages = cache->free_pages;
  a.queue = cache->queue;
  a.queue_out = queue_out_dev;
  a.cu_tokens = plan->cu_tokens;
  a.positions = plan->positions;
  a.runs = plan->runs;
  a.counts = plan->counts;
  a.status = dev_status;
  a.num_rows = num_rows;
  a.num_seqs = cfg->num_seqs;
  a.max_blocks = cfg->max_blocks;
  a.num_pages = cfg->num_pages;
  a.lg_r = log2i(cfg->residual);
  a.max_tokens = plan->max_tokens;
  a.max_runs = plan->max_runs;
  return kivi::launch_tables(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KIVI_OK : KIVI_ERR_CUDA;
}

int kivi_paged_append(const kivi_paged_config* cfg, const kivi_paged_cache* cache, const kivi_paged_plan* plan,
                      const uint16_t* k_dev, const uint16_t* v_dev, int64_t token_stride, int64_t head_stride,
                      int32_t* dev_status, void* stream) {
  const int st = check_paged(cfg);
  if (st != KIVI_OK) return st;
  if (!pool_ok(cache) || plan == nullptr || !aligned16(plan->runs) || !aligned16(plan->counts) || plan->max_tokens < 0 ||
      plan->max_runs < 1 || (plan->max_tokens > 0 && !(aligned16(k_dev) && aligned16(v_dev))) ||
      ((token_stride | head_stride) & 7) != 0 || !status_ok(dev_status))
    return KIVI_ERR_INVALID_ARG;
  const long long runs = plan->max_runs < plan->max_tokens ? plan->max_runs : plan->max_tokens;
  if (runs * cfg->num_kv_heads > 0x7fffffffll) return KIVI_ERR_UNSUPPORTED;
  kivi::PagedAppendArgs a{};
  a.runs = plan->runs;
  a.counts = plan->counts;
  a.k = k_dev;
  a.v = v_dev;
  a.token_stride = token_stride;
  a.head_stride = head_stride;
  a.k_codes = cache->k_codes;
  a.v_codes = cache->v_codes;
  a.k_scale = cache->k_scale;
  a.k_zero = cache->k_zero;
  a.v_scale = cache->v_scale;
  a.v_zero = cache->v_zero;
  a.k_res = cache->k_res;
  a.v_res = cache->v_res;
  a.status = dev_status;
  a.heads = cfg->num_kv_heads;
  a.num_pages = cfg->num_pages;
  a.num_seqs = cfg->num_seqs;
  a.residual = cfg->residual;
  a.lg_gk = log2i(cfg->group_k);
  a.lg_gv = log2i(cfg->group_v);
  a.max_tokens = plan->max_tokens;
  a.max_runs = plan->max_runs;
  return kivi::launch_paged_append(a, cfg->bits, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KIVI_OK : KIVI_ERR_CUDA;
}

size_t kivi_paged_workspace_bytes(const kivi_paged_config* cfg, int32_t num_q_heads) {
  if (check_paged(cfg) != KIVI_OK) return 0;
  return attend_bytes(cfg->num_seqs, cfg->num_kv_heads, num_q_heads, max_units(cfg->bits, cfg->residual, cfg->max_blocks));
}

static int paged_attention(const kivi_paged_config* cfg, const kivi_paged_cache* cache, int32_t num_rows,
                           const int32_t* lens_dev, const int32_t* cu_tokens_dev, const int32_t* positions_dev,
                           int32_t max_tokens, const uint16_t* q_dev, int32_t num_q_rows, int32_t num_q_heads, float scale,
                           int32_t window, int32_t sinks, uint16_t* out_dev, void* workspace_dev, size_t workspace_bytes,
                           int32_t* dev_status, void* stream) {
  int st = check_paged(cfg);
  if (st != KIVI_OK) return st;
  kivi::AttendArgs a{};
  a.positions = positions_dev;
  a.max_tokens = max_tokens;
  if ((st = check_attend(cfg->num_kv_heads, num_q_heads, scale, window, sinks, q_dev, out_dev, dev_status, &a)) != KIVI_OK)
    return st;
  if (!pool_ok(cache) || !aligned16(cache->block_table) || num_rows < 0 || num_rows > cfg->num_seqs || num_q_rows < 0 ||
      (num_rows > 0 && !aligned(lens_dev, 4)) || (cu_tokens_dev != nullptr && !aligned(cu_tokens_dev, 4)))
    return KIVI_ERR_INVALID_ARG;
  if (cu_tokens_dev == nullptr && num_q_rows < num_rows) return KIVI_ERR_INVALID_ARG;
  a.k_codes = cache->k_codes;
  a.v_codes = cache->v_codes;
  a.k_scale = cache->k_scale;
  a.k_zero = cache->k_zero;
  a.v_scale = cache->v_scale;
  a.v_zero = cache->v_zero;
  a.k_res = cache->k_res;
  a.v_res = cache->v_res;
  a.block_table = cache->block_table;
  a.lens = lens_dev;
  a.cu_tokens = cu_tokens_dev;
  a.rows = num_rows;
  a.max_rows = cfg->num_seqs;
  a.q_rows = num_q_rows;
  a.num_pages = cfg->num_pages;
  a.max_blocks = cfg->max_blocks;
  a.lg_r = log2i(cfg->residual);
  a.lg_gk = log2i(cfg->group_k);
  a.lg_gv = log2i(cfg->group_v);
  return run_attend(a, cfg->bits, max_units(cfg->bits, cfg->residual, cfg->max_blocks), workspace_dev, workspace_bytes, stream);
}

int kivi_paged_decode_attention(const kivi_paged_config* cfg, const kivi_paged_cache* cache, int32_t num_rows,
                                const int32_t* lens_dev, const int32_t* cu_tokens_dev, const uint16_t* q_dev,
                                int32_t num_q_rows, int32_t num_q_heads, float scale, int32_t window, int32_t sinks,
                                uint16_t* out_dev, void* workspace_dev, size_t workspace_bytes, int32_t* dev_status,
                                void* stream) {
  return paged_attention(cfg, cache, num_rows, lens_dev, cu_tokens_dev, nullptr, 0, q_dev, num_q_rows, num_q_heads, scale, window,
                         sinks, out_dev, workspace_dev, workspace_bytes, dev_status, stream);
}

int kivi_paged_plan_attention(const kivi_paged_config* cfg, const kivi_paged_cache* cache, const kivi_paged_plan* plan,
                              int32_t num_rows, const int32_t* lens_dev, const uint16_t* q_dev, int32_t num_q_rows,
                              int32_t num_q_heads, float scale, int32_t window, int32_t sinks, uint16_t* out_dev,
                              void* workspace_dev, size_t workspace_bytes, int32_t* dev_status, void* stream) {
  if (plan == nullptr || !aligned16(plan->cu_tokens) || !aligned16(plan->positions) || plan->max_tokens < 1)
    return KIVI_ERR_INVALID_ARG;
  return paged_attention(cfg, cache, num_rows, lens_dev, plan->cu_tokens, plan->positions, plan->max_tokens, q_dev, num_q_rows,
                         num_q_heads, scale, window, sinks, out_dev, workspace_dev, workspace_bytes, dev_status, stream);
}

}  // extern "C"
