// C ABI of libkvq.so: host-side argument validation and the stream-ordered
// launcher (kernel variant and grid from format, head_dim, GQA ratio and
// context length).  No allocation, no per-call state.
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <chrono>

#include "../../include/kvq.h"
#include "kvq_device.cuh"
#include "kvq_internal.h"
#include "rope_turns.h"

using namespace kvq;

namespace {

constexpr float kLog2e = 1.4426950408889634f;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool valid_fmt(int f) { return f >= KVQ_FMT_INT8 && f <= KVQ_FMT_E4M3_BLOCK; }

// Families that share a kernel: per-tensor-scaled 8-bit codes, per-row
// asymmetric codes (optionally KVarN), 8-bit codes scaled per page and kv-head, and the
// 16-bit cache (K and V both).
bool pairing_ok(int kf, int vf, bool kvarn) {
  if ((kf == KVQ_FMT_BF16) != (vf == KVQ_FMT_BF16)) return false;
  if (is_block(kf) != is_block(vf)) return false;
  const bool ak = is_asym(kf), av = is_asym(vf);
  if (kvarn) return ak && av;
  return ak == av;
}
bool scaled(int f) { return !is_asym(f) && !is_block(f) && f != KVQ_FMT_BF16; }
constexpr bool has_meta(int f) { return is_asym(f) || is_block(f); }

// A power of two from 8 to 128: a 16-token tile lies in one block, or in two
// consecutive entries of the block table (8-token pages).
bool supported_block_size(int bs) {
  return bs == 8 || bs == 16 || bs == 32 || bs == 64 || bs == 128;
}

// A range of bytes; two that overlap (empty ones never do).
struct Span {
  const void* p;
  size_t n;
};
bool overlap(const Span& a, const Span& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return a.n > 0 && b.n > 0 && x < y + b.n && y < x + a.n;
}

// Rows of `width` 16-bit elements, `stride` elements apart.
struct Rows {
  const void* p;
  int64_t stride, width;
};
bool rows_ok(const Rows& r) {
  return r.width == 0 || (r.p != nullptr && aligned(r.p, 16) && r.stride >= r.width && r.stride % 8 == 0);
}
// Whether two sets of n rows share a byte; exact for equal strides (slices of
// one packed projection), else whether their address ranges overlap.
bool rows_meet(const Rows& a, const Rows& b, int64_t n) {
  if (a.width == 0 || b.width == 0 || n == 0) return false;
  const Span sa = {a.p, static_cast<size_t>(((n - 1) * a.stride + a.width) * 2)};
  const Span sb = {b.p, static_cast<size_t>(((n - 1) * b.stride + b.width) * 2)};
  if (!overlap(sa, sb)) return false;
  if (a.stride != b.stride || n == 1) return true;
  const int64_t pitch = 2 * a.stride;
  int64_t d = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p)) % pitch;
  if (d < 0) d += pitch;
  return d < 2 * a.width || d + 2 * b.width > pitch;
}

// Checks shared by write and decode on the cache description.
kvq_status check_cache(const kvq_cache_desc* c) {
  if (c == nullptr) return KVQ_ERR_INVALID_ARGUMENT;
  if (!valid_fmt(c->k_fmt) || !valid_fmt(c->v_fmt)) return KVQ_ERR_INVALID_ARGUMENT;
  if (c->num_kv_heads < 1 || c->num_blocks < 1 || c->block_size < 1 || c->head_dim < 1)
    return KVQ_ERR_INVALID_ARGUMENT;
  if (c->flags & ~KVQ_FLAG_VARNORM_ROTATE) return KVQ_ERR_INVALID_ARGUMENT;
  if (c->head_dim != 64 && c->head_dim != 128) return KVQ_ERR_UNSUPPORTED;
  if (!supported_block_size(c->block_size)) return KVQ_ERR_UNSUPPORTED;
  const bool kvarn = (c->flags & KVQ_FLAG_VARNORM_ROTATE) != 0;
  if (!pairing_ok(c->k_fmt, c->v_fmt, kvarn)) return KVQ_ERR_UNSUPPORTED;
  if (scaled(c->k_fmt) && !(c->k_scale > 0.0f && isfinite(c->k_scale)))
    return KVQ_ERR_INVALID_ARGUMENT;
  if (scaled(c->v_fmt) && !(c->v_scale > 0.0f && isfinite(c->v_scale)))
    return KVQ_ERR_INVALID_ARGUMENT;
  if (has_meta(c->k_fmt) && (c->k_meta == nullptr || !aligned(c->k_meta, 16)))
    return KVQ_ERR_INVALID_ARGUMENT;
  if (has_meta(c->v_fmt) && (c->v_meta == nullptr || !aligned(c->v_meta, 16)))
    return KVQ_ERR_INVALID_ARGUMENT;
  if (kvarn && c->signs != nullptr && !aligned(c->signs, 16)) return KVQ_ERR_INVALID_ARGUMENT;
  // per-kv-head scales: scaled symmetric formats only
  if (c->k_head_scales != nullptr && (!scaled(c->k_fmt) || !aligned(c->k_head_scales, 4)))
    return KVQ_ERR_INVALID_ARGUMENT;
  if (c->v_head_scales != nullptr && (!scaled(c->v_fmt) || !aligned(c->v_head_scales, 4)))
    return KVQ_ERR_INVALID_ARGUMENT;
  return KVQ_OK;
}

float rotation_scale(int d) { return static_cast<float>(1.0 / sqrt(static_cast<double>(d))); }

// SM count of the current device, cached per device.
int sm_count() {
  static std::atomic<int> cache[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return -1;
  int v = (dev >= 0 && dev < 64) ? cache[dev].load() : 0;
  if (v > 0) return v;
  if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return -1;
  if (dev >= 0 && dev < 64) cache[dev].store(v);
  return v;
}

int ceil_div(long long a, long long b) { return static_cast<int>((a + b - 1) / b); }

int heads_per_cta(int hkv) { return hkv < 8 ? hkv : 8; }

// Stream-K ranges per head group: as many as the decode kernel has resident
// CTAs (two per SM; one for the 16-bit cache, whose 64 KB stages fill an
// SM's shared memory), at most one per possible tile.
int auto_ctas(int num_seqs, int max_ctx, int head_groups, int sms, int per_sm) {
  const long long tiles_max = static_cast<long long>(num_seqs) * ((max_ctx + 15) / 16);
  long long nc =
      (static_cast<long long>(sms > 0 ? sms : 152) * per_sm + head_groups - 1) / head_groups;
  if (nc > tiles_max) nc = tiles_max;
  if (nc > kMaxCtas) nc = kMaxCtas;
  return static_cast<int>(nc < 1 ? 1 : nc);
}

// Workspace: per (range, head group, first/last segment of the range, head) a
// partial output of D fp16 (acc / l) and its (max, sum) in f32; per (range,
// head group, first/last segment) three 64-bit words (completion tag, team
// tag, team claim); per (sequence, head group) a 64-bit merge claim.  One
// range needs none.
size_t workspace_bytes_for(int num_seqs, int hq, int hkv, int d, int nc) {
  if (nc <= 1) return 0;
  const size_t rows = static_cast<size_t>(nc) * 2 * hq;
  const size_t groups = static_cast<size_t>(hkv / heads_per_cta(hkv));
  return rows * (d * 2 + 2 * sizeof(float)) + static_cast<size_t>(nc) * groups * 2 * 8 * 3 +
         static_cast<size_t>(num_seqs) * groups * 8;
}

// Test hook of the bounded pipeline waits (kvq_debug_arm_wait_timeout): armed
// for the next decode or chunk-attention launch of the process only.
std::atomic<int> g_wait_hook_armed{0};
std::atomic<int> g_wait_hook_polls{0};
std::atomic<int> g_wait_hook_cta{-1};
std::atomic<int> g_wait_hook_tile{-1};

// Polls of an mbarrier before a decode CTA gives up (the kernel's default), and before
// one of the chunk or prompt attention does.  A poll sleeps for up to 3.7 us (measured: 61 ms
// for 2^14), so 15 s and one.
constexpr int kDefaultSpinLimit = 1 << 22;
constexpr int kPrefillSpinLimit = 1 << 18;
// What a launch gets of the hook, and its default.
template <class Args>
void bound_waits(Args* a, int spin_limit) {
  a->spin_limit = spin_limit;
  a->withhold_cta = -1;
  a->withhold_tile = -1;
  if (g_wait_hook_armed.exchange(0) != 0) {
    a->spin_limit = g_wait_hook_polls.load();
    a->withhold_cta = g_wait_hook_cta.load();
    a->withhold_tile = g_wait_hook_tile.load();
  }
}

// Nonzero 64-bit tag, different for every decode call of the process, so that
// the completion tags never need clearing between calls.
unsigned long long next_epoch() {
  static std::atomic<unsigned long long> counter{0};
  static const unsigned long long base = [] {
    unsigned long long x = static_cast<unsigned long long>(
        std::chrono::steady_clock::now().time_since_epoch().count());
    x ^= reinterpret_cast<uintptr_t>(&counter) * 0x9E3779B97F4A7C15ull;
    return x;
  }();
  const unsigned long long e = base + counter.fetch_add(1);
  return e == 0 ? 1 : e;
}

kvq_status decode_shape(const kvq_cache_desc* c, int32_t num_seqs, int32_t num_q_heads,
                        int32_t max_context_len, int32_t num_ctas, int* NC) {
  kvq_status st = check_cache(c);
  if (st != KVQ_OK) return st;
  if (num_seqs < 0 || num_q_heads < 1 || max_context_len < 0) return KVQ_ERR_INVALID_ARGUMENT;
  if (num_q_heads % c->num_kv_heads) return KVQ_ERR_INVALID_ARGUMENT;
  if (num_q_heads / c->num_kv_heads > 8) return KVQ_ERR_UNSUPPORTED;
  if (c->num_kv_heads > 8 && c->num_kv_heads % 8) return KVQ_ERR_UNSUPPORTED;
  if (num_ctas < 0 || num_ctas > kMaxCtas) return KVQ_ERR_INVALID_ARGUMENT;
  int nc = num_ctas;
  if (nc == 0) {
    const int sms = sm_count();
    if (sms <= 0) return KVQ_ERR_CUDA;
    nc = auto_ctas(num_seqs, max_context_len, c->num_kv_heads / heads_per_cta(c->num_kv_heads),
                   sms, c->k_fmt == KVQ_FMT_BF16 ? 1 : 2);
  }
  *NC = nc;
  return KVQ_OK;
}

// Checks shared by the norm and rotation calls; fills what they share of *a.
kvq_status check_rope(const kvq_rope_desc* r, const int32_t* positions, int64_t num_tokens,
                      int32_t num_q_heads, int32_t num_kv_heads, NormRopeArgs* a) {
  if (r == nullptr || num_tokens < 0 || num_q_heads < 0 || num_kv_heads < 0)
    return KVQ_ERR_INVALID_ARGUMENT;
  if (r->head_dim < 1 || r->rot_dim < 0 || r->rot_dim > r->head_dim ||
      (r->interleaved != 0 && r->interleaved != 1) || !(r->eps >= 0.0f) || !isfinite(r->eps) ||
      !isfinite(r->weight_offset))
    return KVQ_ERR_INVALID_ARGUMENT;
  if ((r->head_dim != 64 && r->head_dim != 128 && r->head_dim != 256) || r->rot_dim % 16)
    return KVQ_ERR_UNSUPPORTED;
  if (!aligned(r->q_weight, 16) || !aligned(r->k_weight, 16)) return KVQ_ERR_INVALID_ARGUMENT;
  if (r->rot_dim > 0) {
    if (r->num_positions < 0) return KVQ_ERR_INVALID_ARGUMENT;
    if (num_tokens > 0 && (!r->table || !aligned(r->table, 16) || !positions || !aligned(positions, 4)))
      return KVQ_ERR_INVALID_ARGUMENT;
  }
  a->positions = positions;
  a->table = r->table;
  a->q_weight = static_cast<const uint16_t*>(r->q_weight);
  a->k_weight = static_cast<const uint16_t*>(r->k_weight);
  a->num_positions = r->num_positions;
  a->num_tokens = num_tokens;
  a->num_q_heads = num_q_heads;
  a->num_kv_heads = num_kv_heads;
  a->rot_dim = r->rot_dim;
  a->interleaved = r->interleaved;
  a->eps = r->eps;
  a->weight_offset = r->weight_offset;
  return KVQ_OK;
}

// Row tiles and key splits of a prefill launch.
struct PrefillShape {
  int rows = 128;           // rows of a tile
  int tiles = 0;            // row tiles, of all sequences, that the batch may need
  int splits = 1;
  size_t partial_rows = 0;  // rows of partial results in the workspace
  int staged_len = 0;       // positions of a context dequantized ahead (0: not ahead)
  size_t staged = 0;        // bytes of those, and of the flags behind them
  size_t workspace = 0;
};
// Dequantizing ahead pays where each key is read by this many row tiles (of 256) on
// average, fewer where dequantizing costs more, and is done in at most 16 GiB.
// Measured ahead / not, 32 / 8 heads of 128: int8, 8 x 4,096 keys: 4 row tiles 160 /
// 138 us, 8 257 / 257, 1 x 8,192 keys and 32 tiles 193 / 217; KVarN, 16 x 4,096 keys:
// 2 tiles 223 / 222, 8 x 4,096: 4 tiles 182 / 210, 8 289 / 389; int4 4 tiles 165 / 177;
// bf16 as int8; int8 per page, 8 x 4,096: 4 tiles 168 / 142, 6 221 / 206, 8 270 / 266,
// 32 x 2,048: 6 429 / 411, 8 518 / 518, 1 x 8,192 keys and 32 tiles 203 / 227.
constexpr int64_t stage_tiles(int fmt) { return is_asym(fmt) ? 3 : 8; }
constexpr int64_t kStageBytes = 16ll << 30;
// Bytes of a tile of 128 keys' scales behind them: three float32 for every 8 (block formats).
constexpr size_t stage_scale_bytes(int fmt) { return is_block(fmt) ? 3 * 128 / 8 * 4 : 0; }
// What can be said of a batch's sizes without a device.
kvq_status check_prefill(const kvq_cache_desc* c, int32_t num_seqs, int32_t num_q_heads,
                         int64_t total_q, int32_t max_query_len, int32_t max_context_len) {
  kvq_status st = check_cache(c);
  if (st != KVQ_OK) return st;
  if (num_seqs < 0 || num_q_heads < 1 || total_q < 0 || max_query_len < 0 || max_context_len < 0)
    return KVQ_ERR_INVALID_ARGUMENT;
  if (num_q_heads % c->num_kv_heads) return KVQ_ERR_INVALID_ARGUMENT;
  if (num_q_heads / c->num_kv_heads > 8) return KVQ_ERR_UNSUPPORTED;
  if (total_q > INT32_MAX || max_context_len > (1 << 30)) return KVQ_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(c->block_size) * c->num_kv_heads * c->head_dim * 2 > INT32_MAX)
    return KVQ_ERR_UNSUPPORTED;  // a block's bytes fit 31 bits
  return KVQ_OK;
}
// The launch of a batch that check_prefill has passed.
kvq_status prefill_shape(const kvq_cache_desc* c, int32_t num_seqs, int32_t num_q_heads,
                         int64_t total_q, int32_t max_query_len, int32_t max_context_len,
                         PrefillShape* sh) {
  if (num_seqs == 0 || total_q == 0 || max_query_len == 0) return KVQ_OK;
  const int sms = sm_count();
  if (sms <= 0) return KVQ_ERR_CUDA;
  const int64_t g = num_q_heads / c->num_kv_heads, hkv = c->num_kv_heads;
  sh->rows = max_query_len * g <= 64 ? 64 : max_query_len * g <= 128 ? 128 : 256;
  // no more than every sequence at its longest, nor than the rows there are with
  // a tile per sequence not full
  const int64_t longest = (max_query_len * g + sh->rows - 1) / sh->rows;
  const int64_t tiles = std::min(num_seqs * longest, total_q * g / sh->rows + num_seqs);
  if (tiles * hkv > INT32_MAX) return KVQ_ERR_UNSUPPORTED;
  sh->tiles = static_cast<int>(tiles);
  // too few tiles for the SMs: cut the keys, into parts of two key tiles or more
  const int64_t parts = std::min<int64_t>(sms / (tiles * hkv), (max_context_len + 255) / 256);
  sh->splits = static_cast<int>(std::min<int64_t>(std::max<int64_t>(parts, 1), 64));
  if (sh->splits > 1) {
    sh->partial_rows = static_cast<size_t>(sh->splits) * tiles * hkv * sh->rows;
    sh->workspace = sh->partial_rows * (c->head_dim + 2) * sizeof(float);
  }
  const int64_t len = (max_context_len + 127ll) / 128 * 128, rows = num_seqs * hkv * len;
  if (sh->rows == 256 && total_q * g >= stage_tiles(c->k_fmt) * 256 * num_seqs && 2 * rows <= INT32_MAX &&
      num_seqs * (len / 128) <= INT32_MAX && hkv <= 65535 && 2 * rows * c->head_dim * 2 <= kStageBytes) {
    sh->staged_len = static_cast<int>(len);
    sh->staged = (static_cast<size_t>(2 * rows) * c->head_dim * 2 + rows / 128 * (stage_scale_bytes(c->k_fmt) + 1) + 15) / 16 * 16;
    sh->workspace += sh->staged;
  }
  return KVQ_OK;
}
// A workspace for every batch of at most these sizes, of which the smaller ones can
// need more: fewer row tiles leave more parts to cut the keys into, and fewer
// sequences have more row tiles each, which is when keys are dequantized ahead.
kvq_status prefill_workspace(const kvq_cache_desc* c, int32_t num_seqs, int32_t num_q_heads,
                             int64_t total_q, int32_t max_query_len, int32_t max_context_len,
                             size_t* bytes) {
  PrefillShape sh;
  kvq_status st = prefill_shape(c, num_seqs, num_q_heads, total_q, max_query_len, max_context_len, &sh);
  *bytes = 0;
  if (st != KVQ_OK || sh.tiles == 0) return st;
  const int64_t sms = sm_count(), g = num_q_heads / c->num_kv_heads, hkv = c->num_kv_heads, d = c->head_dim;
  // Partial results: splits * tiles * hkv <= SMs (splits > 1 is a floor of their
  // quotient), of no more rows a tile than these sizes'; and no more splits or rows
  // than there can be.
  const int64_t parts = std::min<int64_t>((max_context_len + 255) / 256, 64);
  if (parts > 1 && 2 * hkv <= sms) {
    const int64_t longest = (max_query_len * g + sh.rows - 1) / sh.rows;
    const int64_t ctas = std::min(std::min(num_seqs * longest, sms) * hkv * parts, sms);
    *bytes = static_cast<size_t>(ctas) * sh.rows * (d + 2) * sizeof(float);
  }
  // Contexts dequantized ahead: of as many sequences as the rows are enough for.
  if (sh.rows == 256 && hkv <= 65535) {
    const int64_t len = (max_context_len + 127ll) / 128 * 128;
    const int64_t seqs = std::min<int64_t>(num_seqs, total_q * g / (stage_tiles(c->k_fmt) * 256));
    const int64_t rows = std::min(std::min<int64_t>(seqs * hkv * len, INT32_MAX / 2), kStageBytes / (4 * d));
    *bytes += (static_cast<size_t>(2 * rows) * d * 2 + rows / 128 * (stage_scale_bytes(c->k_fmt) + 1) + 15) / 16 * 16;
  }
  return KVQ_OK;
}

}  // namespace

extern "C" {

const char* kvq_status_string(kvq_status s) {
  switch (s) {
    case KVQ_OK: return "KVQ_OK";
    case KVQ_ERR_INVALID_ARGUMENT: return "KVQ_ERR_INVALID_ARGUMENT";
    case KVQ_ERR_UNSUPPORTED: return "KVQ_ERR_UNSUPPORTED";
    case KVQ_ERR_WORKSPACE: return "KVQ_ERR_WORKSPACE";
    case KVQ_ERR_CUDA: return "KVQ_ERR_CUDA";
  }
  return "KVQ_ERR_UNKNOWN";
}

const char* kvq_version(void) { return "kvq 0.1.0 sm_103a"; }

kvq_status kvq_write_cache(const kvq_cache_desc* cache, void* k_cache, void* v_cache,
                           const void* key, const void* value, int64_t key_stride,
                           int64_t value_stride, const int64_t* slot_mapping, int64_t num_tokens,
                           kvq_stream_t stream) {
  kvq_status st = check_cache(cache);
  if (st != KVQ_OK) return st;
  if (num_tokens < 0) return KVQ_ERR_INVALID_ARGUMENT;
  if (num_tokens == 0) return KVQ_OK;
  if (!k_cache || !v_cache || !key || !value || !slot_mapping) return KVQ_ERR_INVALID_ARGUMENT;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(key, 16) || !aligned(value, 16) ||
      !aligned(slot_mapping, 8))
    return KVQ_ERR_INVALID_ARGUMENT;
  const int64_t row = static_cast<int64_t>(cache->num_kv_heads) * cache->head_dim;
  if (key_stride < row || value_stride < row || key_stride % 8 || value_stride % 8)
    return KVQ_ERR_INVALID_ARGUMENT;
  if (num_tokens > (1LL << 31) * 8) return KVQ_ERR_UNSUPPORTED;
  const bool kvarn = (cache->flags & KVQ_FLAG_VARNORM_ROTATE) != 0;
  const bool block = is_block(cache->k_fmt);
  const int sms = block ? sm_count() : 0;
  if (block && sms <= 0) return KVQ_ERR_CUDA;
  WriteArgs a;
  a.key = static_cast<const uint16_t*>(key);
  a.value = static_cast<const uint16_t*>(value);
  a.key_stride = key_stride;
  a.value_stride = value_stride;
  a.slot_mapping = slot_mapping;
  a.num_tokens = num_tokens;
  a.k_cache = static_cast<uint8_t*>(k_cache);
  a.v_cache = static_cast<uint8_t*>(v_cache);
  a.k_meta = static_cast<__half*>(cache->k_meta);
  a.v_meta = static_cast<__half*>(cache->v_meta);
  a.num_kv_heads = cache->num_kv_heads;
  a.block_size = cache->block_size;
  a.block_shift = __builtin_ctz(static_cast<unsigned>(cache->block_size));
  a.num_blocks = cache->num_blocks;
  // inv = 1/scale, one IEEE float32 division on the host
  volatile float one = 1.0f;
  a.k_inv = scaled(cache->k_fmt) ? one / cache->k_scale : 1.0f;
  a.v_inv = scaled(cache->v_fmt) ? one / cache->v_scale : 1.0f;
  a.k_head_scale = cache->k_head_scales;
  a.v_head_scale = cache->v_head_scales;
  a.signs = cache->signs;
  a.cR = rotation_scale(cache->head_dim);
  const cudaError_t e =
      block ? launch_write_block(a, AppendSlots{}, cache->head_dim, cache->k_fmt, cache->v_fmt, stream, sms)
            : launch_write(a, cache->head_dim, cache->k_fmt, cache->v_fmt, kvarn, stream);
  if (e == cudaErrorNotSupported) return KVQ_ERR_UNSUPPORTED;
  return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

kvq_status kvq_decode_workspace_size_ex(const kvq_cache_desc* cache, int32_t num_seqs,
                                        int32_t num_q_heads, int32_t max_context_len,
                                        int32_t num_ctas, size_t* bytes) {
  if (bytes == nullptr) return KVQ_ERR_INVALID_ARGUMENT;
  int NC = 0;
  kvq_status st = decode_shape(cache, num_seqs, num_q_heads, max_context_len, num_ctas, &NC);
  if (st != KVQ_OK) return st;
  *bytes = workspace_bytes_for(num_seqs, num_q_heads, cache->num_kv_heads, cache->head_dim, NC);
  return KVQ_OK;
}

kvq_status kvq_decode_workspace_size(const kvq_cache_desc* cache, int32_t num_seqs,
                                     int32_t num_q_heads, int32_t max_context_len,
                                     size_t* bytes) {
  return kvq_decode_workspace_size_ex(cache, num_seqs, num_q_heads, max_context_len, 0, bytes);
}

}  // extern "C"

namespace {

// The new-token rows of kvq_decode_append (nullptr key: a plain decode).
struct AppendRows {
  const void* key = nullptr;
  const void* value = nullptr;
  int64_t key_stride = 0;
  int64_t value_stride = 0;
};

// Page classes of a mixed cache: every class the same formats, kv-heads,
// head_dim, flags, scales and signs as class 0; pages of 16 tokens or more
// (an 8-token page takes its own kernel instance, one page size per call).
kvq_status check_classes(const kvq_cache_desc* classes, int32_t num_classes,
                         void* const* k_caches, void* const* v_caches, const uint8_t* seq_class) {
  if (classes == nullptr || k_caches == nullptr || v_caches == nullptr || seq_class == nullptr)
    return KVQ_ERR_INVALID_ARGUMENT;
  if (num_classes < 1 || num_classes > kMaxPageClasses) return KVQ_ERR_UNSUPPORTED;
  if (is_block(classes[0].k_fmt)) return KVQ_ERR_UNSUPPORTED;  // no such instances: page scales of class 0 only
  const kvq_cache_desc& c0 = classes[0];
  for (int c = 0; c < num_classes; ++c) {
    const kvq_cache_desc& x = classes[c];
    kvq_status st = check_cache(&x);
    if (st != KVQ_OK) return st;
    if (x.k_fmt != c0.k_fmt || x.v_fmt != c0.v_fmt || x.num_kv_heads != c0.num_kv_heads ||
        x.head_dim != c0.head_dim || x.flags != c0.flags || x.signs != c0.signs ||
        x.k_head_scales != c0.k_head_scales || x.v_head_scales != c0.v_head_scales ||
        (scaled(x.k_fmt) && x.k_scale != c0.k_scale) || (scaled(x.v_fmt) && x.v_scale != c0.v_scale))
      return KVQ_ERR_INVALID_ARGUMENT;
    if (x.block_size < 16) return KVQ_ERR_UNSUPPORTED;
    if (k_caches[c] == nullptr || v_caches[c] == nullptr || !aligned(k_caches[c], 16) ||
        !aligned(v_caches[c], 16))
      return KVQ_ERR_INVALID_ARGUMENT;
  }
  return KVQ_OK;
}

kvq_status decode_call(const kvq_cache_desc* classes, int32_t num_classes,
                       void* const* k_caches, void* const* v_caches, const uint8_t* seq_class,
                       void* out, const void* query, int32_t num_seqs, int32_t num_q_heads,
                       const int32_t* block_table, int32_t max_blocks_per_seq,
                       const int32_t* context_lens, int32_t max_context_len, float sm_scale,
                       int32_t num_ctas, void* workspace, size_t workspace_bytes,
                       const AppendRows& app, kvq_stream_t stream, int32_t window = 0,
                       int32_t num_sinks = 0) {
  const kvq_cache_desc* cache = classes;  // class 0: formats, heads, scales of every class
  int NC = 0;
  kvq_status st = decode_shape(cache, num_seqs, num_q_heads, max_context_len, num_ctas, &NC);
  if (st != KVQ_OK) return st;
  if (num_seqs == 0) return KVQ_OK;
  if (!k_caches[0] || !v_caches[0] || !out || !query || !block_table || !context_lens)
    return KVQ_ERR_INVALID_ARGUMENT;
  if (!aligned(k_caches[0], 16) || !aligned(v_caches[0], 16) || !aligned(out, 16) ||
      !aligned(query, 16) || !aligned(block_table, 4) || !aligned(context_lens, 4))
    return KVQ_ERR_INVALID_ARGUMENT;
  int min_bs = cache->block_size;
  for (int c = 1; c < num_classes; ++c)
    min_bs = classes[c].block_size < min_bs ? classes[c].block_size : min_bs;
  if (max_blocks_per_seq < ceil_div(max_context_len, min_bs) || max_blocks_per_seq < 0)
    return KVQ_ERR_INVALID_ARGUMENT;
  if (!isfinite(sm_scale)) return KVQ_ERR_INVALID_ARGUMENT;
  const size_t need =
      workspace_bytes_for(num_seqs, num_q_heads, cache->num_kv_heads, cache->head_dim, NC);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return KVQ_ERR_WORKSPACE;
  if (need > 0 && !aligned(workspace, 16)) return KVQ_ERR_INVALID_ARGUMENT;
  const bool kvarn = (cache->flags & KVQ_FLAG_VARNORM_ROTATE) != 0;
  DecodeArgs a;
  const bool append = app.key != nullptr;
  for (int c = 0; c < kMaxPageClasses; ++c) {
    const int cc = c < num_classes ? c : 0;
    const kvq_cache_desc& x = classes[cc];
    a.k_cache[c] = static_cast<const uint8_t*>(k_caches[cc]);
    a.v_cache[c] = static_cast<const uint8_t*>(v_caches[cc]);
    a.k_meta[c] = static_cast<const __half*>(x.k_meta);
    a.v_meta[c] = static_cast<const __half*>(x.v_meta);
    a.block_shift[c] = __builtin_ctz(static_cast<unsigned>(x.block_size));
    a.num_blocks[c] = x.num_blocks;
    a.k_cache_w[c] = append ? static_cast<uint8_t*>(k_caches[cc]) : nullptr;
    a.v_cache_w[c] = append ? static_cast<uint8_t*>(v_caches[cc]) : nullptr;
    a.k_meta_w[c] = append ? static_cast<__half*>(x.k_meta) : nullptr;
    a.v_meta_w[c] = append ? static_cast<__half*>(x.v_meta) : nullptr;
  }
  a.seq_class = seq_class;
  a.num_classes = num_classes;
  a.query = static_cast<const uint16_t*>(query);
  a.out = static_cast<uint16_t*>(out);
  a.block_table = block_table;
  a.context_lens = context_lens;
  a.signs = cache->signs;
  const size_t rows = static_cast<size_t>(NC) * 2 * num_q_heads;
  a.ws_acc = need ? static_cast<__half*>(workspace) : nullptr;
  a.ws_ml = need ? reinterpret_cast<float*>(static_cast<__half*>(workspace) + rows * cache->head_dim)
                 : nullptr;
  a.tags = need ? reinterpret_cast<unsigned long long*>(a.ws_ml + rows * 2) : nullptr;
  const size_t slot_words = static_cast<size_t>(NC) *
                           (cache->num_kv_heads / heads_per_cta(cache->num_kv_heads)) * 2;
  a.team_tags = need ? a.tags + slot_words : nullptr;
  a.team_claims = need ? a.tags + 2 * slot_words : nullptr;
  a.claims = need ? a.tags + 3 * slot_words : nullptr;
  a.epoch = next_epoch();
  a.num_seqs = num_seqs;
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = cache->num_kv_heads;
  a.gqa = num_q_heads / cache->num_kv_heads;
  a.heads_per_cta = heads_per_cta(cache->num_kv_heads);
  a.max_blocks_per_seq = max_blocks_per_seq;
  a.max_context_len = max_context_len;
  a.num_ctas = NC;
  a.window = window;
  a.sinks = num_sinks;
  a.qk_scale = sm_scale * kLog2e * (scaled(cache->k_fmt) ? cache->k_scale : 1.0f);
  a.v_scale = scaled(cache->v_fmt) ? cache->v_scale : 1.0f;
  a.qk_base = sm_scale * kLog2e;
  a.k_head_scale = cache->k_head_scales;
  a.v_head_scale = cache->v_head_scales;
  a.cR = rotation_scale(cache->head_dim);
  a.new_key = static_cast<const uint16_t*>(app.key);
  a.new_value = static_cast<const uint16_t*>(app.value);
  a.new_key_stride = app.key_stride;
  a.new_value_stride = app.value_stride;
  volatile float one = 1.0f;  // 1/scale, one IEEE float32 division, as kvq_write_cache
  a.k_inv = scaled(cache->k_fmt) ? one / cache->k_scale : 1.0f;
  a.v_inv = scaled(cache->v_fmt) ? one / cache->v_scale : 1.0f;
  bound_waits(&a, kDefaultSpinLimit);
  // A launch recorded into a CUDA graph is replayed with the same call tag, so
  // a replay would find the tags and claims its predecessor left: while the
  // stream is capturing, the call first clears them (a memset node that runs
  // before the kernel at every replay).  Direct calls take a fresh tag instead.
  if (need > 0) {
    cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(static_cast<cudaStream_t>(stream), &cap) != cudaSuccess)
      return KVQ_ERR_CUDA;
    if (cap == cudaStreamCaptureStatusActive) {
      const size_t words = 3 * slot_words + static_cast<size_t>(num_seqs) *
                                                (cache->num_kv_heads / heads_per_cta(cache->num_kv_heads));
      if (cudaMemsetAsync(a.tags, 0, words * sizeof(unsigned long long),
                          static_cast<cudaStream_t>(stream)) != cudaSuccess)
        return KVQ_ERR_CUDA;
    }
  }
  cudaError_t e = cudaErrorNotSupported;
  const int kf = cache->k_fmt, vf = cache->v_fmt;
  if (append && is_block(kf)) {  // the new rows first: one may change its page's scale and codes
    const int sms = sm_count();
    if (sms <= 0) return KVQ_ERR_CUDA;
    WriteArgs w = {};
    w.key = a.new_key;
    w.value = a.new_value;
    w.key_stride = a.new_key_stride;
    w.value_stride = a.new_value_stride;
    w.num_tokens = num_seqs;
    w.k_cache = a.k_cache_w[0];
    w.v_cache = a.v_cache_w[0];
    w.k_meta = a.k_meta_w[0];
    w.v_meta = a.v_meta_w[0];
    w.num_kv_heads = cache->num_kv_heads;
    w.block_size = cache->block_size;
    w.block_shift = a.block_shift[0];
    w.num_blocks = cache->num_blocks;
    e = launch_write_block(w, AppendSlots{block_table, context_lens, max_blocks_per_seq, max_context_len},
                           cache->head_dim, kf, vf, stream, sms);
    if (e != cudaSuccess) return e == cudaErrorNotSupported ? KVQ_ERR_UNSUPPORTED : KVQ_ERR_CUDA;
  }
#define KVQ_UNIT_LAUNCHER(U) launch_##U,
  static const DecodeLauncher launchers[] = {KVQ_DECODE_UNITS(KVQ_UNIT_LAUNCHER)};
#undef KVQ_UNIT_LAUNCHER
  for (DecodeLauncher f : launchers) {  // the unit that holds the instance launches it
    e = f(a, cache->head_dim, kf, vf, kvarn, stream);
    if (e != cudaErrorNotSupported) break;
  }
  if (e == cudaErrorNotSupported) return KVQ_ERR_UNSUPPORTED;
  return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

// The new-token rows of kvq_decode_append, checked.
kvq_status append_rows(const kvq_cache_desc* cache, int32_t num_seqs, const void* new_key,
                       const void* new_value, int64_t key_stride, int64_t value_stride,
                       AppendRows* app) {
  if (num_seqs > 0) {
    if (!new_key || !new_value || !aligned(new_key, 16) || !aligned(new_value, 16))
      return KVQ_ERR_INVALID_ARGUMENT;
    const int64_t row = static_cast<int64_t>(cache->num_kv_heads) * cache->head_dim;
    if (key_stride < row || value_stride < row || key_stride % 8 || value_stride % 8)
      return KVQ_ERR_INVALID_ARGUMENT;
    if (!is_block(cache->k_fmt) &&
        !write_supported(cache->k_fmt, cache->v_fmt, (cache->flags & KVQ_FLAG_VARNORM_ROTATE) != 0))
      return KVQ_ERR_UNSUPPORTED;
  }
  app->key = new_key;
  app->value = new_value;
  app->key_stride = key_stride;
  app->value_stride = value_stride;
  return KVQ_OK;
}

}  // namespace

extern "C" {

kvq_status kvq_paged_decode_ex(const kvq_cache_desc* cache, const void* k_cache,
                               const void* v_cache, void* out, const void* query,
                               int32_t num_seqs, int32_t num_q_heads, const int32_t* block_table,
                               int32_t max_blocks_per_seq, const int32_t* context_lens,
                               int32_t max_context_len, float sm_scale, int32_t num_ctas,
                               void* workspace, size_t workspace_bytes, kvq_stream_t stream) {
  void* kc = const_cast<void*>(k_cache);
  void* vc = const_cast<void*>(v_cache);
  return decode_call(cache, 1, &kc, &vc, nullptr, out, query, num_seqs, num_q_heads, block_table,
                     max_blocks_per_seq, context_lens, max_context_len, sm_scale, num_ctas,
                     workspace, workspace_bytes, AppendRows{}, stream);
}

kvq_status kvq_decode_append(const kvq_cache_desc* cache, void* k_cache, void* v_cache,
                             const void* new_key, const void* new_value, int64_t key_stride,
                             int64_t value_stride, void* out, const void* query,
                             int32_t num_seqs, int32_t num_q_heads, const int32_t* block_table,
                             int32_t max_blocks_per_seq, const int32_t* context_lens,
                             int32_t max_context_len, float sm_scale, int32_t num_ctas,
                             void* workspace, size_t workspace_bytes, kvq_stream_t stream) {
  kvq_status st = check_cache(cache);
  if (st != KVQ_OK) return st;
  AppendRows app;
  st = append_rows(cache, num_seqs, new_key, new_value, key_stride, value_stride, &app);
  if (st != KVQ_OK) return st;
  return decode_call(cache, 1, &k_cache, &v_cache, nullptr, out, query, num_seqs, num_q_heads,
                     block_table, max_blocks_per_seq, context_lens, max_context_len, sm_scale,
                     num_ctas, workspace, workspace_bytes, app, stream);
}

kvq_status kvq_decode_mixed(const kvq_cache_desc* classes, int32_t num_classes,
                            void* const* k_caches, void* const* v_caches,
                            const uint8_t* seq_class, const void* new_key, const void* new_value,
                            int64_t key_stride, int64_t value_stride, void* out,
                            const void* query, int32_t num_seqs, int32_t num_q_heads,
                            const int32_t* block_table, int32_t max_blocks_per_seq,
                            const int32_t* context_lens, int32_t max_context_len,
                            float sm_scale, int32_t num_ctas, void* workspace,
                            size_t workspace_bytes, kvq_stream_t stream) {
  kvq_status st = check_classes(classes, num_classes, k_caches, v_caches, seq_class);
  if (st != KVQ_OK) return st;
  AppendRows app;
  if (new_key != nullptr || new_value != nullptr) {
    st = append_rows(classes, num_seqs, new_key, new_value, key_stride, value_stride, &app);
    if (st != KVQ_OK) return st;
  }
  return decode_call(classes, num_classes, k_caches, v_caches, seq_class, out, query, num_seqs,
                     num_q_heads, block_table, max_blocks_per_seq, context_lens,
                     max_context_len, sm_scale, num_ctas, workspace, workspace_bytes, app,
                     stream);
}

kvq_status kvq_decode_window(const kvq_cache_desc* cache, void* k_cache, void* v_cache,
                             const void* new_key, const void* new_value, int64_t key_stride,
                             int64_t value_stride, void* out, const void* query, int32_t num_seqs,
                             int32_t num_q_heads, const int32_t* block_table,
                             int32_t max_blocks_per_seq, const int32_t* context_lens,
                             int32_t max_context_len, float sm_scale, int32_t window,
                             int32_t num_sinks, int32_t num_ctas, void* workspace,
                             size_t workspace_bytes, kvq_stream_t stream) {
  kvq_status st = check_cache(cache);
  if (st != KVQ_OK) return st;
  if (window < 1 || num_sinks < 0) return KVQ_ERR_INVALID_ARGUMENT;
  AppendRows app;
  if (new_key != nullptr || new_value != nullptr) {
    st = append_rows(cache, num_seqs, new_key, new_value, key_stride, value_stride, &app);
    if (st != KVQ_OK) return st;
  }
  return decode_call(cache, 1, &k_cache, &v_cache, nullptr, out, query, num_seqs, num_q_heads,
                     block_table, max_blocks_per_seq, context_lens, max_context_len, sm_scale,
                     num_ctas, workspace, workspace_bytes, app, stream, window, num_sinks);
}

kvq_status kvq_paged_decode(const kvq_cache_desc* cache, const void* k_cache,
                            const void* v_cache, void* out, const void* query, int32_t num_seqs,
                            int32_t num_q_heads, const int32_t* block_table,
                            int32_t max_blocks_per_seq, const int32_t* context_lens,
                            int32_t max_context_len, float sm_scale, void* workspace,
                            size_t workspace_bytes, kvq_stream_t stream) {
  return kvq_paged_decode_ex(cache, k_cache, v_cache, out, query, num_seqs, num_q_heads,
                             block_table, max_blocks_per_seq, context_lens, max_context_len,
                             sm_scale, 0, workspace, workspace_bytes, stream);
}

kvq_status kvq_plan_step(const int32_t* context_lens, const int32_t* new_lens, int32_t num_seqs,
                         int32_t* block_table, int32_t max_blocks_per_seq, int32_t block_size,
                         int32_t num_blocks, const int32_t* free_blocks, int32_t free_capacity,
                         const int32_t* free_range, int64_t* slot_mapping, int32_t* positions,
                         int64_t max_tokens, int32_t* context_lens_out, int32_t* cu_new,
                         int32_t* free_range_out, kvq_stream_t stream) {
  if (num_seqs < 0 || max_blocks_per_seq < 0 || block_size < 1 || num_blocks < 1 ||
      free_capacity < 0 || max_tokens < 0)
    return KVQ_ERR_INVALID_ARGUMENT;
  if (!supported_block_size(block_size)) return KVQ_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(max_blocks_per_seq) * block_size > (1 << 30) || max_tokens > INT32_MAX)
    return KVQ_ERR_UNSUPPORTED;
  if (!free_range || !free_range_out || !cu_new) return KVQ_ERR_INVALID_ARGUMENT;
  if (num_seqs > 0 && (!context_lens || !new_lens || !context_lens_out ||
                       (max_blocks_per_seq > 0 && !block_table)))
    return KVQ_ERR_INVALID_ARGUMENT;
  if ((free_capacity > 0 && !free_blocks) || (max_tokens > 0 && (!slot_mapping || !positions)))
    return KVQ_ERR_INVALID_ARGUMENT;
  for (const void* p : {static_cast<const void*>(context_lens), static_cast<const void*>(new_lens),
                        static_cast<const void*>(block_table), static_cast<const void*>(free_blocks),
                        static_cast<const void*>(free_range), static_cast<const void*>(context_lens_out),
                        static_cast<const void*>(cu_new), static_cast<const void*>(free_range_out)})
    if (!aligned(p, 4)) return KVQ_ERR_INVALID_ARGUMENT;
  if (!aligned(slot_mapping, 16) || !aligned(positions, 16)) return KVQ_ERR_INVALID_ARGUMENT;
  // every CTA reads the inputs while others write: nothing written may be read
  const size_t n = static_cast<size_t>(num_seqs), t = static_cast<size_t>(max_tokens);
  const Span out[] = {{slot_mapping, 8 * t},
                      {positions, 4 * t},
                      {context_lens_out, 4 * n},
                      {cu_new, 4 * n + 4},
                      {free_range_out, 8},
                      {block_table, 4 * n * static_cast<size_t>(max_blocks_per_seq)}};
  const Span in[] = {{context_lens, 4 * n},
                     {new_lens, 4 * n},
                     {free_blocks, 4 * static_cast<size_t>(free_capacity)},
                     {free_range, 8}};
  for (int i = 0; i < 6; ++i) {
    for (int j = i + 1; j < 6; ++j)
      if (overlap(out[i], out[j])) return KVQ_ERR_INVALID_ARGUMENT;
    for (const Span& x : in)
      if (overlap(out[i], x)) return KVQ_ERR_INVALID_ARGUMENT;
  }
  PlanArgs a;
  a.context_lens = context_lens;
  a.new_lens = new_lens;
  a.block_table = block_table;
  a.free_blocks = free_blocks;
  a.free_range = free_range;
  a.slot_mapping = slot_mapping;
  a.positions = positions;
  a.context_lens_out = context_lens_out;
  a.cu_new = cu_new;
  a.free_range_out = free_range_out;
  a.max_tokens = max_tokens;
  a.num_seqs = num_seqs;
  a.max_blocks_per_seq = max_blocks_per_seq;
  a.block_shift = __builtin_ctz(static_cast<unsigned>(block_size));
  a.num_blocks = num_blocks;
  a.free_capacity = free_capacity;
  return launch_plan(a, stream) == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

kvq_status kvq_rope_table(float* table, int64_t num_positions, int32_t rot_dim, double base,
                          const kvq_rope_scaling* scaling, kvq_stream_t stream) {
  if (num_positions < 0 || rot_dim < 2 || rot_dim % 2 || !(base > 1.0) || !isfinite(base))
    return KVQ_ERR_INVALID_ARGUMENT;
  if (rot_dim > 2 * kMaxRopePairs || num_positions > INT32_MAX) return KVQ_ERR_UNSUPPORTED;
  const kvq_rope_scaling none = {KVQ_ROPE_NONE, 1.0, 1.0, 1.0, 2.0, 1.0};
  const kvq_rope_scaling& sc = scaling ? *scaling : none;
  if (sc.kind < KVQ_ROPE_NONE || sc.kind > KVQ_ROPE_BANDS || !isfinite(sc.amplitude))
    return KVQ_ERR_INVALID_ARGUMENT;
  if (sc.kind != KVQ_ROPE_NONE && !(sc.factor > 0.0 && isfinite(sc.factor)))
    return KVQ_ERR_INVALID_ARGUMENT;
  if (sc.kind == KVQ_ROPE_NTK && rot_dim == 2) return KVQ_ERR_INVALID_ARGUMENT;
  if (sc.kind >= KVQ_ROPE_YARN &&
      !(sc.original_len > 0.0 && isfinite(sc.original_len) && sc.low > 0.0 && sc.high > sc.low &&
        isfinite(sc.high)))
    return KVQ_ERR_INVALID_ARGUMENT;
  RopeTurns turns;
  if (!rope_turns(rot_dim, base, sc, &turns)) return KVQ_ERR_INVALID_ARGUMENT;
  if (num_positions == 0) return KVQ_OK;
  if (!table || !aligned(table, 16)) return KVQ_ERR_INVALID_ARGUMENT;
  const int sms = sm_count();
  if (sms <= 0) return KVQ_ERR_CUDA;
  const cudaError_t e = launch_rope_table(table, num_positions, rot_dim / 2,
                                          static_cast<float>(sc.amplitude), turns, stream, sms);
  return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

kvq_status kvq_norm_rope(const kvq_rope_desc* rope, void* query_out, int64_t query_out_stride,
                         void* key_out, int64_t key_out_stride, const void* query,
                         int64_t query_stride, const void* key, int64_t key_stride,
                         const int32_t* positions, int64_t num_tokens, int32_t num_q_heads,
                         int32_t num_kv_heads, kvq_stream_t stream) {
  NormRopeArgs a = {};
  kvq_status st = check_rope(rope, positions, num_tokens, num_q_heads, num_kv_heads, &a);
  if (st != KVQ_OK || num_tokens == 0 || num_q_heads + num_kv_heads == 0) return st;
  const int d = rope->head_dim;
  const Rows rows[] = {{query, query_stride, num_q_heads * static_cast<int64_t>(d)},
                       {key, key_stride, num_kv_heads * static_cast<int64_t>(d)},
                       {query_out, query_out_stride, num_q_heads * static_cast<int64_t>(d)},
                       {key_out, key_out_stride, num_kv_heads * static_cast<int64_t>(d)}};
  for (const Rows& r : rows)
    if (!rows_ok(r)) return KVQ_ERR_INVALID_ARGUMENT;
  for (int o = 2; o < 4; ++o)  // outputs against inputs (in place allowed) and each other
    for (int i = 0; i < o; ++i) {
      const bool in_place = i == o - 2 && rows[i].p == rows[o].p && rows[i].stride == rows[o].stride;
      if (!in_place && rows_meet(rows[o], rows[i], num_tokens)) return KVQ_ERR_INVALID_ARGUMENT;
    }
  a.query = static_cast<const uint16_t*>(query);
  a.key = static_cast<const uint16_t*>(key);
  a.query_out = static_cast<uint16_t*>(query_out);
  a.key_out = static_cast<uint16_t*>(key_out);
  a.query_stride = query_stride;
  a.key_stride = key_stride;
  a.query_out_stride = query_out_stride;
  a.key_out_stride = key_out_stride;
  const cudaError_t e = launch_norm_rope(a, d, stream);
  if (e == cudaErrorNotSupported) return KVQ_ERR_UNSUPPORTED;
  return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

kvq_status kvq_norm_rope_write(const kvq_rope_desc* rope, const kvq_cache_desc* cache, void* k_cache,
                               void* v_cache, void* query_out, int64_t query_out_stride,
                               const void* query, int64_t query_stride, const void* key,
                               int64_t key_stride, const void* value, int64_t value_stride,
                               const int32_t* positions, const int64_t* slot_mapping,
                               int64_t num_tokens, int32_t num_q_heads, kvq_stream_t stream) {
  kvq_status st = check_cache(cache);
  if (st != KVQ_OK) return st;
  NormRopeArgs a = {};
  st = check_rope(rope, positions, num_tokens, num_q_heads, cache->num_kv_heads, &a);
  if (st != KVQ_OK) return st;
  if (rope->head_dim != cache->head_dim) return KVQ_ERR_INVALID_ARGUMENT;
  if (is_block(cache->k_fmt)) return KVQ_ERR_UNSUPPORTED;  // kvq_norm_rope, then kvq_write_cache
  if (num_tokens == 0) return KVQ_OK;
  const int64_t d = cache->head_dim, row = cache->num_kv_heads * d;
  if (!k_cache || !v_cache || !slot_mapping || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(slot_mapping, 8))
    return KVQ_ERR_INVALID_ARGUMENT;
  const Rows rows[] = {{query, query_stride, num_q_heads * d}, {key, key_stride, row},
                       {value, value_stride, row}, {query_out, query_out_stride, num_q_heads * d}};
  for (const Rows& r : rows)
    if (!rows_ok(r)) return KVQ_ERR_INVALID_ARGUMENT;
  for (int i = 0; i < 3; ++i) {
    const bool in_place = i == 0 && query == query_out && query_stride == query_out_stride;
    if (!in_place && rows_meet(rows[3], rows[i], num_tokens)) return KVQ_ERR_INVALID_ARGUMENT;
  }
  a.query = static_cast<const uint16_t*>(query);
  a.key = static_cast<const uint16_t*>(key);
  a.value = static_cast<const uint16_t*>(value);
  a.query_out = static_cast<uint16_t*>(query_out);
  a.query_stride = query_stride;
  a.key_stride = key_stride;
  a.value_stride = value_stride;
  a.query_out_stride = query_out_stride;
  a.slot_mapping = slot_mapping;
  a.k_cache = static_cast<uint8_t*>(k_cache);
  a.v_cache = static_cast<uint8_t*>(v_cache);
  a.k_meta = static_cast<__half*>(cache->k_meta);
  a.v_meta = static_cast<__half*>(cache->v_meta);
  a.block_size = cache->block_size;
  a.block_shift = __builtin_ctz(static_cast<unsigned>(cache->block_size));
  a.num_blocks = cache->num_blocks;
  volatile float one = 1.0f;  // 1/scale, one IEEE float32 division, as kvq_write_cache
  a.k_inv = scaled(cache->k_fmt) ? one / cache->k_scale : 1.0f;
  a.v_inv = scaled(cache->v_fmt) ? one / cache->v_scale : 1.0f;
  a.k_head_scale = cache->k_head_scales;
  a.v_head_scale = cache->v_head_scales;
  a.signs = cache->signs;
  a.cR = rotation_scale(cache->head_dim);
  const cudaError_t e = launch_norm_rope_write(a, cache->head_dim, cache->k_fmt, cache->v_fmt,
                                               (cache->flags & KVQ_FLAG_VARNORM_ROTATE) != 0, stream);
  if (e == cudaErrorNotSupported) return KVQ_ERR_UNSUPPORTED;
  return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

kvq_status kvq_prefill_workspace_size(const kvq_cache_desc* cache, int32_t num_seqs,
                                      int32_t num_q_heads, int64_t total_q, int32_t max_query_len,
                                      int32_t max_context_len, size_t* bytes) {
  if (bytes == nullptr) return KVQ_ERR_INVALID_ARGUMENT;
  kvq_status st = check_prefill(cache, num_seqs, num_q_heads, total_q, max_query_len, max_context_len);
  if (st != KVQ_OK) return st;
  size_t n = 0;
  st = prefill_workspace(cache, num_seqs, num_q_heads, total_q, max_query_len, max_context_len, &n);
  if (st != KVQ_OK) return st;
  *bytes = n;
  return KVQ_OK;
}

kvq_status kvq_paged_prefill(const kvq_cache_desc* cache, const void* k_cache, const void* v_cache,
                             void* out, const void* query, const int32_t* cu_query,
                             int32_t num_seqs, int64_t total_q, int32_t max_query_len,
                             int32_t num_q_heads, const int32_t* block_table,
                             int32_t max_blocks_per_seq, const int32_t* context_lens,
                             int32_t max_context_len, float sm_scale, int32_t window,
                             int32_t num_sinks, void* workspace, size_t workspace_bytes,
                             kvq_stream_t stream) {
  kvq_status st = check_prefill(cache, num_seqs, num_q_heads, total_q, max_query_len, max_context_len);
  if (st != KVQ_OK) return st;
  if (window < 0 || num_sinks < 0 || !isfinite(sm_scale)) return KVQ_ERR_INVALID_ARGUMENT;
  if (num_seqs == 0 || total_q == 0 || max_query_len == 0) return KVQ_OK;
  if (!k_cache || !v_cache || !out || !query || !cu_query || !block_table || !context_lens)
    return KVQ_ERR_INVALID_ARGUMENT;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) || !aligned(query, 16) ||
      !aligned(cu_query, 4) || !aligned(block_table, 4) || !aligned(context_lens, 4))
    return KVQ_ERR_INVALID_ARGUMENT;
  const size_t rows = static_cast<size_t>(total_q) * num_q_heads * cache->head_dim * 2;
  if (overlap({out, rows}, {query, rows})) return KVQ_ERR_INVALID_ARGUMENT;
  if (max_blocks_per_seq < ceil_div(max_context_len, cache->block_size))
    return KVQ_ERR_INVALID_ARGUMENT;
  PrefillShape sh;  // asks for the device's SMs: after all that the host can refuse by itself
  st = prefill_shape(cache, num_seqs, num_q_heads, total_q, max_query_len, max_context_len, &sh);
  if (st != KVQ_OK) return st;
  if (sh.workspace > 0 && (workspace == nullptr || workspace_bytes < sh.workspace))
    return KVQ_ERR_WORKSPACE;
  if (sh.workspace > 0 && !aligned(workspace, 16)) return KVQ_ERR_INVALID_ARGUMENT;
  PrefillArgs a;
  a.k_cache = static_cast<const uint8_t*>(k_cache);
  a.v_cache = static_cast<const uint8_t*>(v_cache);
  a.k_meta = static_cast<const __half*>(cache->k_meta);
  a.v_meta = static_cast<const __half*>(cache->v_meta);
  a.k_fmt = cache->k_fmt;
  a.v_fmt = cache->v_fmt;
  a.kvarn = (cache->flags & KVQ_FLAG_VARNORM_ROTATE) != 0;
  a.block_shift = __builtin_ctz(static_cast<unsigned>(cache->block_size));
  a.num_blocks = cache->num_blocks;
  a.query = static_cast<const uint16_t*>(query);
  a.out = static_cast<uint16_t*>(out);
  a.cu_query = cu_query;
  a.block_table = block_table;
  a.context_lens = context_lens;
  a.signs = cache->signs;
  a.k_head_scale = cache->k_head_scales;
  a.v_head_scale = cache->v_head_scales;
  a.k_scale = scaled(cache->k_fmt) ? cache->k_scale : 1.0f;
  a.v_scale = scaled(cache->v_fmt) ? cache->v_scale : is_block(cache->v_fmt) ? kSumUnit : 1.0f;  // over the row's sum
  a.sm_scale_log2 = sm_scale * kLog2e;
  a.cR = rotation_scale(cache->head_dim);
  a.num_seqs = num_seqs;
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = cache->num_kv_heads;
  a.gqa = num_q_heads / cache->num_kv_heads;
  a.total_q = total_q;
  a.max_query_len = max_query_len;
  a.max_blocks_per_seq = max_blocks_per_seq;
  a.max_context_len = max_context_len;
  a.window = std::min(window, 1 << 30);  // contexts are no longer
  a.sinks = std::min(num_sinks, 1 << 30);
  a.rows_per_tile = sh.rows;
  a.tiles = sh.tiles;
  a.num_splits = sh.splits;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.staged = sh.staged ? reinterpret_cast<uint16_t*>(ws) : nullptr;
  a.staged_len = sh.staged_len;
  const size_t staged_rows = static_cast<size_t>(num_seqs) * cache->num_kv_heads * sh.staged_len;
  uint8_t* const behind = ws + 2 * staged_rows * cache->head_dim * 2;
  a.staged_scales = reinterpret_cast<float*>(behind);
  a.staged_bad = behind + staged_rows / 128 * stage_scale_bytes(cache->k_fmt);
  a.ws_out = reinterpret_cast<float*>(ws + sh.staged);
  a.ws_ml = a.ws_out + sh.partial_rows * cache->head_dim;
  bound_waits(&a, kPrefillSpinLimit);
  const cudaError_t e = launch_prefill(a, cache->head_dim, stream);
  if (e == cudaErrorNotSupported) return KVQ_ERR_UNSUPPORTED;
  return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

kvq_status kvq_prompt_attention(void* out, int64_t out_stride, const void* query, int64_t query_stride,
                                const void* key, int64_t key_stride, const void* value,
                                int64_t value_stride, const int32_t* cu_seqlens, int32_t num_seqs,
                                int64_t total_tokens, int32_t max_len, int32_t num_q_heads,
                                int32_t num_kv_heads, int32_t head_dim, float sm_scale, int32_t window,
                                int32_t num_sinks, kvq_stream_t stream) {
  if (num_seqs < 0 || total_tokens < 0 || max_len < 0 || num_q_heads < 1 || num_kv_heads < 1 ||
      head_dim < 1 || window < 0 || num_sinks < 0 || !isfinite(sm_scale))
    return KVQ_ERR_INVALID_ARGUMENT;
  if (num_q_heads % num_kv_heads) return KVQ_ERR_INVALID_ARGUMENT;
  if (num_q_heads / num_kv_heads > 8 || (head_dim != 64 && head_dim != 128)) return KVQ_ERR_UNSUPPORTED;
  if (total_tokens > (1 << 30)) return KVQ_ERR_UNSUPPORTED;
  if (num_seqs == 0 || total_tokens == 0 || max_len == 0) return KVQ_OK;
  const int64_t d = head_dim;
  const Rows rows[] = {{query, query_stride, num_q_heads * d}, {key, key_stride, num_kv_heads * d},
                       {value, value_stride, num_kv_heads * d}, {out, out_stride, num_q_heads * d}};
  for (const Rows& r : rows)
    if (!rows_ok(r) || r.stride > (1ll << 31)) return KVQ_ERR_INVALID_ARGUMENT;
  if (!cu_seqlens || !aligned(cu_seqlens, 4)) return KVQ_ERR_INVALID_ARGUMENT;
  for (int i = 0; i < 3; ++i)  // other CTAs read what one writes: not in place
    if (rows_meet(rows[3], rows[i], total_tokens)) return KVQ_ERR_INVALID_ARGUMENT;
  const int sms = sm_count();
  if (sms <= 0) return KVQ_ERR_CUDA;
  PromptArgs a = {};
  a.query = static_cast<const uint16_t*>(query);
  a.key = static_cast<const uint16_t*>(key);
  a.value = static_cast<const uint16_t*>(value);
  a.out = static_cast<uint16_t*>(out);
  a.query_stride = query_stride;
  a.key_stride = key_stride;
  a.value_stride = value_stride;
  a.out_stride = out_stride;
  a.cu_seqlens = cu_seqlens;
  a.num_seqs = num_seqs;
  a.total = total_tokens;
  a.max_len = static_cast<int>(std::min<int64_t>(max_len, total_tokens));
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = num_kv_heads;
  a.gqa = num_q_heads / num_kv_heads;
  a.sm_scale_log2 = sm_scale * kLog2e;
  a.window = std::min(window, 1 << 30);  // prompts are no longer
  a.sinks = std::min(num_sinks, 1 << 30);
  bound_waits(&a, kPrefillSpinLimit);
  const cudaError_t e = launch_prompt(a, head_dim, stream, sms);
  if (e == cudaErrorNotSupported) return KVQ_ERR_UNSUPPORTED;
  return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

kvq_status kvq_read_cache(const kvq_cache_desc* cache, const void* k_cache, const void* v_cache,
                          void* key_out, void* value_out, int64_t key_out_stride,
                          int64_t value_out_stride, const int64_t* slot_mapping, int64_t num_tokens,
                          kvq_stream_t stream) {
  kvq_status st = check_cache(cache);
  if (st != KVQ_OK) return st;
  if (num_tokens < 0) return KVQ_ERR_INVALID_ARGUMENT;
  if (num_tokens == 0) return KVQ_OK;
  if (!k_cache || !v_cache || !slot_mapping || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(slot_mapping, 8))
    return KVQ_ERR_INVALID_ARGUMENT;
  const int64_t row = static_cast<int64_t>(cache->num_kv_heads) * cache->head_dim;
  if (num_tokens > (1LL << 31) * 8 || row > INT32_MAX) return KVQ_ERR_UNSUPPORTED;
  const Rows rows[] = {{key_out, key_out_stride, row}, {value_out, value_out_stride, row}};
  if (!rows_ok(rows[0]) || !rows_ok(rows[1]) || rows_meet(rows[0], rows[1], num_tokens))
    return KVQ_ERR_INVALID_ARGUMENT;
  const int sms = sm_count();
  if (sms <= 0) return KVQ_ERR_CUDA;
  ReadArgs a = {};
  a.codes[0] = static_cast<const uint8_t*>(k_cache);
  a.codes[1] = static_cast<const uint8_t*>(v_cache);
  a.meta[0] = cache->k_meta;
  a.meta[1] = cache->v_meta;
  a.head_scale[0] = cache->k_head_scales;
  a.head_scale[1] = cache->v_head_scales;
  a.scale[0] = cache->k_scale;
  a.scale[1] = cache->v_scale;
  a.fmt[0] = cache->k_fmt;
  a.fmt[1] = cache->v_fmt;
  a.out[0] = static_cast<uint16_t*>(key_out);
  a.out[1] = static_cast<uint16_t*>(value_out);
  a.out_stride[0] = key_out_stride;
  a.out_stride[1] = value_out_stride;
  a.slot_mapping = slot_mapping;
  a.num_tokens = num_tokens;
  a.signs = cache->signs;
  a.cR = rotation_scale(cache->head_dim);
  a.num_kv_heads = cache->num_kv_heads;
  a.block_shift = __builtin_ctz(static_cast<unsigned>(cache->block_size));
  a.num_blocks = cache->num_blocks;
  const cudaError_t e =
      launch_read(a, cache->head_dim, (cache->flags & KVQ_FLAG_VARNORM_ROTATE) != 0, stream, sms);
  if (e == cudaErrorNotSupported) return KVQ_ERR_UNSUPPORTED;
  return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

kvq_status kvq_hadamard(void* x, int32_t dtype, int64_t rows, int32_t head_dim,
                        const int8_t* signs, int32_t inverse, kvq_stream_t stream) {
  if (rows < 0 || (dtype != 0 && dtype != 1) || (inverse != 0 && inverse != 1))
    return KVQ_ERR_INVALID_ARGUMENT;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return KVQ_ERR_UNSUPPORTED;
  if (rows == 0) return KVQ_OK;
  if (x == nullptr || !aligned(x, 16)) return KVQ_ERR_INVALID_ARGUMENT;
  if (signs != nullptr && !aligned(signs, 16)) return KVQ_ERR_INVALID_ARGUMENT;
  const cudaError_t e =
      launch_hadamard(x, dtype, rows, head_dim, signs, inverse, rotation_scale(head_dim), stream);
  return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

kvq_status kvq_calibrate_scale(const void* x, int64_t n, float qmax, float* scale_out,
                               kvq_stream_t stream) {
  if (n < 0 || !(qmax > 0.0f && isfinite(qmax)) || scale_out == nullptr ||
      !aligned(scale_out, 4))
    return KVQ_ERR_INVALID_ARGUMENT;
  if (n > 0 && (x == nullptr || !aligned(x, 16))) return KVQ_ERR_INVALID_ARGUMENT;
  const int sms = sm_count();
  if (sms <= 0) return KVQ_ERR_CUDA;
  const cudaError_t e =
      launch_calibrate(static_cast<const uint16_t*>(x), n, qmax, scale_out, stream, sms);
  return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

kvq_status kvq_calibrate_head_scales(const void* x, int64_t num_tokens, int32_t num_kv_heads,
                                     int32_t head_dim, int64_t stride, float qmax,
                                     float* scales_out, kvq_stream_t stream) {
  if (num_tokens < 0 || num_kv_heads < 1 || head_dim < 8 || head_dim % 8 ||
      !(qmax > 0.0f && isfinite(qmax)) || scales_out == nullptr || !aligned(scales_out, 4))
    return KVQ_ERR_INVALID_ARGUMENT;
  if (stride < static_cast<int64_t>(num_kv_heads) * head_dim || stride % 8)
    return KVQ_ERR_INVALID_ARGUMENT;
  if (num_tokens > 0 && (x == nullptr || !aligned(x, 16))) return KVQ_ERR_INVALID_ARGUMENT;
  const int sms = sm_count();
  if (sms <= 0) return KVQ_ERR_CUDA;
  const cudaError_t e =
      launch_calibrate_heads(static_cast<const uint16_t*>(x), num_tokens, num_kv_heads, head_dim,
                             stride, qmax, scales_out, stream, sms);
  return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

kvq_status kvq_debug_arm_wait_timeout(int32_t polls, int32_t cta, int32_t tile) {
  if (polls < 1 || cta < -1 || tile < -1) return KVQ_ERR_INVALID_ARGUMENT;
  g_wait_hook_polls.store(polls);
  g_wait_hook_cta.store(cta);
  g_wait_hook_tile.store(tile);
  g_wait_hook_armed.store(1);
  return KVQ_OK;
}

kvq_status kvq_get_device_error(kvq_stream_t stream, uint32_t* bits) {
  if (bits == nullptr) return KVQ_ERR_INVALID_ARGUMENT;
  if (cudaStreamSynchronize(stream) != cudaSuccess) return KVQ_ERR_CUDA;
  unsigned v = 0;
#define KVQ_UNIT_TAKE(U) take_error_bits_##U,
  cudaError_t (*take[])(unsigned*) = {take_error_bits_write, take_error_bits_write_asym,
                                      take_error_bits_plan, take_error_bits_norm_rope,
                                      take_error_bits_norm_rope_asym, take_error_bits_prefill,
                                      take_error_bits_write_block, take_error_bits_read,
                                      take_error_bits_prompt,
                                      KVQ_DECODE_UNITS(KVQ_UNIT_TAKE)};
#undef KVQ_UNIT_TAKE
  for (auto f : take)
    if (f(&v) != cudaSuccess) return KVQ_ERR_CUDA;
  *bits = v;
  return KVQ_OK;
}

}  // extern "C"
