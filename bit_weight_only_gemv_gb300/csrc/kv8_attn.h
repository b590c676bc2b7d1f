// Host interface between the attention entry (kv8_attn.cu) and the
// prompt-chunk kernel (kv8_chunk.cu).
#pragma once

#include "kv8.cuh"
#include "tc_common.cuh"

namespace w4 {
namespace kv8 {

// Query rows on a key head from which a call takes the prompt-chunk kernel.
// Measured, row tiles of 8 or 16 in the token kernel against tiles of 128: 64
// rows of 128-channel heads on 2 x 8k keys 45 and 55 us, 96 rows 61 and 55, 128
// rows 76 and 57; of 256-channel heads on 4 x 4k keys 32 rows 39 and 54, 64 rows 62 and 55.
constexpr long long chunk_rows(int D) { return D == 256 ? 49 : 81; }

// The tensor map of one side's codes: bytes [page][head][token][channel], boxes of
// `rows` tokens by 128 channels (64 for 64-channel heads), swizzled.
bool tensor_map(CUtensorMap* m, uint8_t* codes, const Cache& c, int rows);

struct ChunkArgs {
  __nv_bfloat16* out;
  float* lse;
  const __nv_bfloat16* q;
  long long q_stride;
  int Hq;
  float scale;
  int window;
  int32_t* status;
};

struct WeighParams {
  CUtensorMap tm;   // of the keys (single tokens) or the query rows (many rows)
  Cache c;
  Batch bt;
  const __nv_bfloat16* q;
  long long q_stride;
  const float* lse;
  int Hq, G;
  float scale;
  int window;
  const int32_t* sel;     // chosen pages (single tokens), or NULL
  const int32_t* n_sel;
  int max_sel;
  int32_t* status;
};

// w4_kv8_weigh for many query rows on a key head (kv8_weigh_tc.cu).
w4_status weigh_many(WeighParams& p, int sms, int dev, w4_stream_t stream);

size_t chunk_workspace_bytes(const Cache& c, const Batch& b, int G, int sms);
w4_status chunk_attn(const Cache& c, const Batch& b, const ChunkArgs& a, void* workspace,
                     int sms, int dev, w4_stream_t stream);

}  // namespace kv8
}  // namespace w4
