// kv8_launch.h -- internal host-side launchers of the 8-bit key/value cache.
// Each returns hipSuccess or the launch error; argument checks happen in
// kv8_api.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kv {

constexpr int kF32 = 0, kBF16 = 1, kF16 = 2;  // KV8_F32, KV8_BF16, KV8_F16

struct Cache {
  int8_t *k, *v;
  float *ks, *vs;
  int32_t n_pages, n_kv, d;
  int page_log, block_log;  // log2 of page_size and block
};

struct Batch {
  const int32_t *table, *lens, *starts;  // starts: NULL, one row a sequence
  int32_t n_seq, n_tok, width, max_new, max_len;
};

// A strided [n_tok][heads][d] array.
struct Rows {
  const void *p;
  int64_t token_stride, head_stride;
  int type;
  bool wide;  // every row starts on a 16-byte border
};

// kv8_write.hip
hipError_t launch_write(const Cache &c, const Batch &b, const Rows &k, const Rows &v, hipStream_t s);
hipError_t launch_read(const Cache &c, const Batch &b, void *k, void *v, int type, hipStream_t s);

struct Attention {
  void *out;
  Rows q;
  int out_type, n_q, group;  // group: query heads of a key/value head
  int window;                // 0: none
  float scale;
  const float *sinks;
  float *lse;
};

// Partial results of a split over the keys: normalized outputs fp32
// [split][n_tok][n_q][d], then their log2 sums [split][n_tok][n_q].
struct Plan {
  bool tiled;  // kv8_tile.hip, or kv8_stream.hip
  int splits;
};
constexpr int64_t kMaxJoinRows = 1 << 20;  // rows that the join of splits is launched for
Plan attention_plan(const Cache &c, const Batch &b, int n_q, int window, bool halves, size_t ws_bytes);
size_t partial_bytes(const Cache &c, const Batch &b, int n_q, int splits);

// kv8_tile.hip; tile_rows: query rows of a workgroup
int tile_rows(int d, bool halves);
hipError_t launch_tile(const Cache &c, const Batch &b, const Attention &a, int splits, void *ws, hipStream_t s);

// kv8_stream.hip
hipError_t launch_stream(const Cache &c, const Batch &b, const Attention &a, int splits, void *ws, hipStream_t s);
// out and lse of the partial results.
hipError_t launch_join(const Cache &c, const Batch &b, const Attention &a, int splits, const void *ws, hipStream_t s);

}  // namespace kv
