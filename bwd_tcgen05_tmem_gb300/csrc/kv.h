// kv.h -- parameter blocks and launchers of the operators around the attention
// kernels: the norm and rotation of queries and keys (qknorm.cu), the page plan
// and the 4-bit cache (kvcache.cu) and attention over it (kvdecode.cu).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

namespace attn {

// Quotients by a number known at launch: n / d for 0 <= n < 2^31, d >= 1
// (Granlund and Montgomery: multiply by ceil(2^(32 + s) / d), s = ceil(log2 d)).
struct FastDiv {
  uint32_t d, mul, shift;
  static FastDiv of(uint32_t d) {
    FastDiv f;
    f.d = d;
    uint32_t s = 0;
    while ((1ull << s) < d) ++s;
    f.shift = s;
    f.mul = (uint32_t)(((1ull << 32) * ((1ull << s) - d)) / d + 1);
    return f;
  }
#ifdef __CUDACC__
  __device__ __forceinline__ uint32_t div(uint32_t n) const {
    const uint32_t t = __umulhi(n, mul);
    return (uint32_t)(((uint64_t)t + n) >> shift);
  }
#endif
};

struct QkSide {  // queries or keys
  const void* x;
  const void* dz;  // backward: the gradient of the rotated rows
  void* out;       // forward: the rotated rows; backward: the gradient of x
  const void* w;   // the norm's weights, or null
  int64_t x_b, x_t, x_h, dz_b, dz_t, dz_h, o_b, o_t, o_h;
  int heads;
  int per_job;     // tokens of a job (above 1 where a token's heads leave lanes idle)
  float* dw;       // backward: [d], or null
};

struct QkParams {
  QkSide side[2];
  const float *cos, *sin;     // [max_pos][rot / 2]
  const int32_t* positions;   // [batch][seqlen] or null
  int batch, seqlen, d, rot, inter, norm, w_f32, max_pos;
  float eps;
  float* partial;             // backward: [blocks][d] partial sums of dw
  FastDiv seq_div, runs[2];   // by seqlen; by the runs of heads of a token
  int blocks[2];              // blocks that work on each side
  int* status;
};

cudaError_t launch_qk_fwd(QkParams& p, bool bf16, int num_sms, cudaStream_t st);
// blocks of the backward for each side (fills p.blocks); false: too many rows
bool qk_bwd_blocks(QkParams& p, int num_sms);
cudaError_t launch_qk_bwd(const QkParams& p, bool bf16, cudaStream_t st);

struct PlanParams {
  const int32_t *ctx, *fresh, *free_pages, *free_head;
  int32_t* table;
  int32_t *cu, *seq, *pos, *slots, *free_head_out;
  int64_t table_stride;
  int batch, cols, page_shift, num_pages, rows, n_free;
  int* status;
};
constexpr int kPlanMaxBatch = 8192;  // 12 bytes of shared memory each
cudaError_t launch_kv_plan(const PlanParams& p, int num_sms, cudaStream_t st);

struct Kv4 {  // the cache
  uint8_t *k_codes, *v_codes;
  uint16_t *k_scales, *v_scales;
  int num_pages, page_size, page_shift, heads, d_qk, d_v;
};

struct KvRowsParams {  // rows stored into or read from the cache
  Kv4 c;
  void *k, *v;  // [tokens][heads][d]
  int64_t k_t, k_h, v_t, v_h;
  const int32_t* slots;
  int tokens;
  FastDiv per_token, vec_k, vec_v;  // 8-element vectors of a token, of a K row, of a V row
  int* status;
};
cudaError_t launch_kv4_write(const KvRowsParams& p, bool bf16, int num_sms, cudaStream_t st);
cudaError_t launch_kv4_read(const KvRowsParams& p, bool bf16, int num_sms, cudaStream_t st);

struct DecodeParams {
  Kv4 c;
  const void* q;
  void* o;
  float* lse;  // [batch][heads_q][seqlen_q]
  const int32_t *table, *seq_lens;
  int64_t q_b, q_t, q_h, o_b, o_t, o_h, table_stride;
  int batch, seqlen_q, heads_q, group, cols, window_left, sinks;
  int rows, row_blocks;  // query rows of a kv head (seqlen_q * group), and blocks of them
  FastDiv by_group, by_blocks;  // by group; by row_blocks
  float scale_log2;
  int o_f32;
  int* info;       // per item: the first and the last run that work on it
  int* ends;       // per run: the item of others that it ends, or -1
  float* partial;  // per run: two pieces of items
  int* status;
};
// Tiles of query columns (8 each) that one block of a call takes.
int decode_col_tiles(int rows, int d_v);
int decode_blocks(const DecodeParams& p, int num_sms);
size_t decode_runs(int blocks);
size_t decode_partial_floats(int blocks, int rows_per_block, int d_v);
cudaError_t launch_kv4_decode(const DecodeParams& p, bool bf16, int blocks, cudaStream_t st);

}  // namespace attn
