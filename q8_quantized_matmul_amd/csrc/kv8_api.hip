// kv8_api.hip -- the C ABI of include/kv8.h: host-side argument checks and
// launches on the caller's stream.  Nothing here allocates device memory.
#include <math.h>
#include <stdint.h>

#include "kv8.h"
#include "kv8_launch.h"
#include "launch.h"

static_assert(KV8_F32 == kv::kF32 && KV8_BF16 == kv::kBF16 && KV8_F16 == kv::kF16,
              "header and library agree on the element types");

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool type_ok(int32_t t) { return t == KV8_F32 || t == KV8_BF16 || t == KV8_F16; }
int type_size(int32_t t) { return t == KV8_F32 ? 4 : 2; }
int status_of(hipError_t e) { return e == hipSuccess ? Q8_0_OK : Q8_0_ELAUNCH; }

// log2 of a power of two in [lo, hi], or -1.
int log_of(int64_t v, int64_t lo, int64_t hi) {
  if (v < lo || v > hi || (v & (v - 1)) != 0) return -1;
  int n = 0;
  while ((int64_t{1} << n) < v) ++n;
  return n;
}

constexpr int64_t kMaxLen = 1 << 30;  // positions, and the tiles fetched ahead of them, in 32 bits
constexpr int64_t kMaxSeq = 1 << 20, kMaxTok = 1 << 24, kMaxStride = int64_t{1} << 40;
// A launch has fewer than 2^32 threads: attention makes a workgroup of 256 for 16 rows and head.
constexpr int64_t kMaxRows = int64_t{1} << 27, kMaxSeqHeads = int64_t{1} << 22;
constexpr int32_t kMaxKvHeads = 4096, kMaxHeads = 1 << 14;

int read_cache(const kv8_cache *c, kv::Cache *out) {
  if (!c || c->n_pages < 1 || c->n_pages > INT32_MAX || c->n_kv < 1 || c->n_kv > kMaxKvHeads) return Q8_0_EINVAL;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 192 && c->head_dim != 256 && c->head_dim != 512)
    return Q8_0_EINVAL;
  const int page_log = log_of(c->page_size, 16, 1024);
  const int block_log = page_log < 0 ? -1 : log_of(c->block, 16, c->page_size < 128 ? c->page_size : 128);
  if (block_log < 0) return Q8_0_EINVAL;
  *out = {static_cast<int8_t *>(c->k_codes), static_cast<int8_t *>(c->v_codes), c->k_scales, c->v_scales,
          (int32_t)c->n_pages, c->n_kv, c->head_dim, page_log, block_log};
  return Q8_0_OK;
}

int read_batch(const kv8_batch *b, const kv::Cache &c, kv::Batch *out) {
  if (!b || b->n_seq < 0 || b->n_seq > kMaxSeq || b->n_tok < 0 || b->n_tok > kMaxTok || b->table_width < 0 ||
      b->table_width > (kMaxLen >> c.page_log) || b->max_new < 0 || b->max_len < 0 || b->n_seq * c.n_kv > kMaxSeqHeads)
    return Q8_0_EINVAL;
  if (!b->starts && b->n_tok != b->n_seq) return Q8_0_EINVAL;
  const int64_t room = b->table_width << c.page_log;
  const int64_t max_new = b->starts ? (b->max_new < b->n_tok ? b->max_new : b->n_tok) : 1;
  const int64_t max_len = b->max_len && b->max_len < room ? b->max_len : room;
  *out = {b->page_table, b->lens, b->starts, (int32_t)b->n_seq, (int32_t)b->n_tok, (int32_t)b->table_width,
          (int32_t)max_new, (int32_t)max_len};
  return Q8_0_OK;
}

bool nothing_to_do(const kv::Batch &b) { return b.n_seq == 0 || b.n_tok == 0 || b.max_new == 0; }

// Pointers of a cache and a batch with work to do.
int check_pointers(const kv::Cache &c, const kv::Batch &b) {
  if (!c.k || !c.v || !c.ks || !c.vs || !b.lens || (!b.table && b.width > 0)) return Q8_0_EINVAL;
  if (!aligned(c.k, 16) || !aligned(c.v, 16) || !aligned(c.ks, 4) || !aligned(c.vs, 4) || !aligned(b.table, 4) ||
      !aligned(b.lens, 4) || !aligned(b.starts, 4))
    return Q8_0_EALIGN;
  return Q8_0_OK;
}

int read_rows(const void *p, int64_t token_stride, int64_t head_stride, int32_t type, kv::Rows *out) {
  if (!type_ok(type) || token_stride < 0 || head_stride < 0 || token_stride > kMaxStride || head_stride > kMaxStride)
    return Q8_0_EINVAL;
  if (!p) return Q8_0_EINVAL;
  if (!aligned(p, type_size(type))) return Q8_0_EALIGN;
  const int per16 = 16 / type_size(type);
  *out = {p, token_stride, head_stride, type,
          aligned(p, 16) && token_stride % per16 == 0 && head_stride % per16 == 0};
  return Q8_0_OK;
}

}  // namespace

namespace kv {

size_t partial_bytes(const Cache &c, const Batch &b, int n_q, int splits) {
  return splits > 1 ? (size_t)splits * b.n_tok * n_q * (c.d + 1) * sizeof(float) : 0;
}

// Which kernel, and how many splits: the least of the estimated times.  Measured, in us:
//   stream: a workgroup takes `alone` for 16 rows and 128 keys where it has a compute unit to itself, and a unit
//     gives one every `shared` where it has several;
//   tiled: a unit takes `tile` for `keys` keys of all its rows, `at_once` workgroups beside each other.
// Both take some us before the first key and behind the last, the join of splits some more, and its traffic.
// What the estimates decide, measured (us, whole calls, stream / tiled): heads of 128, 8 of them, groups of 4: 256
// tokens 10 / 21; 2 x 1000 tokens 75 / 46; 40 sequences of 32 tokens over 2000 keys 133 / 146; 8192 tokens
// 1369 / 562.  Heads of 512, 64 on one, 2 x 300 tokens over 4000 keys 956 / 798; 12 single tokens over up
// to 6000 keys in four and eight splits 58 / 75.  Splits of the stream kernel, one sequence of 2000 keys, 1 / 4 / 16:
// 21 / 13 / 11; of 131072 keys, 16 / 64: 99 / 59; of 64 sequences of up to 8192, 1 / 4: 135 / 140.  Splits of the
// tiled kernel, 512 tokens over 32768 keys, 1 / 2 / 4 / 8: 900 / 467 / 284 / 300 (stream, without splits, 715); 2048
// over 16384, 1 / 2: 515 / 524.
struct Cost {
  float alone, shared, tile;
  int keys, at_once;
};
Cost cost_of(int d, bool halves) {
  const float more = halves ? 1.2f : 1.f;
  switch (d) {
    case 64: return {0.9f * more, 0.5f * more, 2.2f * more, 64, 2};
    case 128: return {1.2f * more, 0.75f * more, 2.4f * more, 64, 1};
    case 192: return {1.6f * more, 1.1f * more, 2.2f * more, 32, 1};
    case 256: return {2.0f * more, 1.55f * more, 2.6f * more, 32, 1};
    default: return {3.0f * more, 3.0f * more, 2.2f * more, 32, 1};
  }
}

Plan attention_plan(const Cache &c, const Batch &b, int n_q, int window, bool halves, size_t ws_bytes) {
  constexpr float kUnits = 256.f, kEnds = 5.f, kTileEnds = 10.f, kJoin = 4.f, kJoinBytes = 4e6f;  // bytes a us
  const Cost cost = cost_of(c.d, halves);
  const int group = n_q / c.n_kv;
  const int64_t most_rows = (int64_t)b.max_new * group;
  // Workgroups launched for tiles of `rows` rows: each sequence's last ones share none, so some find no rows.
  // The tiled kernel starts those first and they are gone when the others need their units; the stream
  // kernel's lie between the others (12 tokens of 64 heads on one: 60 launched, 48 with rows; 4 splits 52 us, 5 62).
  auto launched = [&](int rows) {
    return most_rows > rows ? (int64_t)b.n_tok * group / rows + b.n_seq : b.n_seq;
  };
  auto with_rows = [&](int rows) {
    const int64_t all = (most_rows / rows + (most_rows % rows != 0)) * b.n_seq;
    return all < launched(rows) ? all : launched(rows);
  };
  // keys of the longest row tile, and of a mean one: rows of a prompt see half of it
  float longest = (float)b.max_len;
  if (window && (float)window + (float)b.max_new < longest) longest = (float)window + (float)b.max_new;
  const bool prompt = 2.f * (float)b.max_new > longest;
  const float mean = prompt ? longest - 0.5f * fminf((float)b.max_new, longest) : longest;  // max_new may be any bound

  Plan best{false, 1};
  float least = INFINITY;
  const float streams = (float)(launched(16) * c.n_kv);
  const bool many = (int64_t)b.n_tok * n_q > kMaxJoinRows;
  const int units = (b.max_len + 127) / 128;  // of 128 keys, a step of a workgroup's four waves
  for (int each = units; each >= 1; each -= each > 8 ? (each + 7) / 8 : 1) {
    const int splits = (units + each - 1) / each;
    if (splits > 256 || (many && splits > 1)) break;
    const size_t bytes = partial_bytes(c, b, n_q, splits);
    if (bytes > ws_bytes) continue;  // (fp32 does not hold every size: the kernels would write past the workspace)
    const float rounds = prompt ? fmaxf(1.f, streams * splits / kUnits) : ceilf(streams * splits / kUnits);
    const float t = fminf((float)each, ceilf(mean / 128.f)) * fmaxf(cost.alone, cost.shared * rounds) + kEnds * fmaxf(1.f, rounds / 4.f) +
                    (splits > 1 ? kJoin + 2.f * (float)bytes / kJoinBytes : 0.f);
    if (t < least) {
      least = t;
      best.splits = splits;
    }
  }
  if (!(halves && c.d > 256)) {  // its operands do not fit the registers
    const float tiles = (float)(with_rows(tile_rows(c.d, halves)) * c.n_kv);
    for (int splits = 1; splits <= 64 && (splits == 1 || (!many && splits <= units)); ++splits) {
      const size_t bytes = partial_bytes(c, b, n_q, splits);
      if (bytes > ws_bytes) break;
      const float each = tiles * splits / (kUnits * cost.at_once);
      const float rounds = prompt ? fmaxf(1.f, each) : ceilf(each);
      const float one = cost.tile / (cost.keys * (float)splits);
      const float t = fmaxf(longest * one + kTileEnds, rounds * (mean * one + kTileEnds)) +
                      (splits > 1 ? kJoin + 2.f * (float)bytes / kJoinBytes : 0.f);
      if (t < least) {
        least = t;
        best = {true, splits};
      }
    }
  }
  return best;
}

}  // namespace kv

namespace {

// kernel: KV8_KERNEL_AUTO, or the one to run with `splits` splits (0: one).
int run_attention(const kv8_cache *cache, const kv8_batch *batch, const kv8_attention_args *args, void *workspace,
                  size_t workspace_bytes, int32_t kernel, int32_t splits, hipStream_t stream) {
  kv::Cache c;
  kv::Batch b;
  int st = read_cache(cache, &c);
  if (st == Q8_0_OK) st = read_batch(batch, c, &b);
  if (st != Q8_0_OK || !args) return Q8_0_EINVAL;
  const kv8_attention_args &x = *args;
  if (x.n_q < 1 || x.n_q > kMaxHeads || x.n_q % c.n_kv != 0 || x.window < 0 || !isfinite(x.scale) ||
      !type_ok(x.out_type) || !type_ok(x.q_type) || (int64_t)b.n_tok * x.n_q > kMaxRows)
    return Q8_0_EINVAL;
  const bool halves = x.q_type == KV8_F32 || x.out_type == KV8_F32;
  if (kernel < KV8_KERNEL_AUTO || kernel > KV8_KERNEL_TILED || splits < 0 || splits > 256 ||
      (kernel == KV8_KERNEL_AUTO && splits != 0) || (kernel == KV8_KERNEL_TILED && halves && c.d > 256) ||
      (splits > 1 && (int64_t)b.n_tok * x.n_q > kv::kMaxJoinRows))
    return Q8_0_EINVAL;
  if (nothing_to_do(b)) return Q8_0_OK;
  // a window of all positions is none (and a position below 0 less a larger one would leave 32 bits)
  const int32_t window = x.window < kMaxLen ? x.window : 0;
  kv::Attention a{x.out, {}, x.out_type, x.n_q, x.n_q / c.n_kv, window, x.scale, x.sinks, x.lse};
  if ((st = check_pointers(c, b)) != Q8_0_OK || (st = read_rows(x.q, x.q_token_stride, x.q_head_stride, x.q_type, &a.q)) != Q8_0_OK)
    return st;
  if (!x.out) return Q8_0_EINVAL;
  if (!aligned(x.out, 16) || !aligned(x.sinks, 4) || !aligned(x.lse, 4) || !aligned(workspace, 16)) return Q8_0_EALIGN;
  if (!workspace) workspace_bytes = 0;
  kv::Plan p{kernel == KV8_KERNEL_TILED, splits > 1 ? splits : 1};
  if (kernel == KV8_KERNEL_AUTO)
    p = kv::attention_plan(c, b, x.n_q, window, halves, workspace_bytes);
  else if (kv::partial_bytes(c, b, x.n_q, p.splits) > workspace_bytes)
    return Q8_0_EWORKSPACE;
  if ((st = q8::check_device()) != Q8_0_OK) return st;
  hipError_t e = p.tiled ? kv::launch_tile(c, b, a, p.splits, workspace, stream)
                         : kv::launch_stream(c, b, a, p.splits, workspace, stream);
  if (e == hipSuccess && p.splits > 1) e = kv::launch_join(c, b, a, p.splits, workspace, stream);
  return status_of(e);
}

}  // namespace

extern "C" {

int kv8_write(const kv8_cache *cache, const kv8_batch *batch, const void *k, int64_t k_token_stride,
              int64_t k_head_stride, const void *v, int64_t v_token_stride, int64_t v_head_stride,
              int32_t type, hipStream_t stream) {
  kv::Cache c;
  kv::Batch b;
  kv::Rows kr, vr;
  int st = read_cache(cache, &c);
  if (st == Q8_0_OK) st = read_batch(batch, c, &b);
  if (st != Q8_0_OK || !type_ok(type)) return Q8_0_EINVAL;
  if (nothing_to_do(b)) return Q8_0_OK;
  if ((st = check_pointers(c, b)) != Q8_0_OK || (st = read_rows(k, k_token_stride, k_head_stride, type, &kr)) != Q8_0_OK ||
      (st = read_rows(v, v_token_stride, v_head_stride, type, &vr)) != Q8_0_OK)
    return st;
  if ((st = q8::check_device()) != Q8_0_OK) return st;
  return status_of(kv::launch_write(c, b, kr, vr, stream));
}

int kv8_read(const kv8_cache *cache, const kv8_batch *batch, void *k, void *v, int32_t type,
             hipStream_t stream) {
  kv::Cache c;
  kv::Batch b;
  int st = read_cache(cache, &c);
  if (st == Q8_0_OK) st = read_batch(batch, c, &b);
  if (st != Q8_0_OK || !type_ok(type)) return Q8_0_EINVAL;
  if (nothing_to_do(b) || (!k && !v)) return Q8_0_OK;
  if ((st = check_pointers(c, b)) != Q8_0_OK) return st;
  if (!aligned(k, 16) || !aligned(v, 16)) return Q8_0_EALIGN;
  if ((st = q8::check_device()) != Q8_0_OK) return st;
  return status_of(kv::launch_read(c, b, k, v, type, stream));
}

size_t kv8_attention_workspace_bytes(const kv8_cache *cache, const kv8_batch *batch, int32_t n_q) {
  kv::Cache c;
  kv::Batch b;
  if (read_cache(cache, &c) != Q8_0_OK || read_batch(batch, c, &b) != Q8_0_OK || n_q < 1 || n_q > kMaxHeads ||
      n_q % c.n_kv != 0 || (int64_t)b.n_tok * n_q > kMaxRows || nothing_to_do(b))
    return 0;
  size_t most = 0;
  for (bool halves : {false, true}) {
    const kv::Plan p = kv::attention_plan(c, b, n_q, 0, halves, SIZE_MAX);
    const size_t bytes = kv::partial_bytes(c, b, n_q, p.splits);
    if (bytes > most) most = bytes;
  }
  return most;
}

int kv8_attention(const kv8_cache *cache, const kv8_batch *batch, const kv8_attention_args *args,
                  void *workspace, size_t workspace_bytes, hipStream_t stream) {
  return run_attention(cache, batch, args, workspace, workspace_bytes, KV8_KERNEL_AUTO, 0, stream);
}

int kv8_attention_debug(const kv8_cache *cache, const kv8_batch *batch, const kv8_attention_args *args,
                        void *workspace, size_t workspace_bytes, int32_t kernel, int32_t splits,
                        hipStream_t stream) {
  return run_attention(cache, batch, args, workspace, workspace_bytes, kernel, splits, stream);
}

}  // extern "C"
