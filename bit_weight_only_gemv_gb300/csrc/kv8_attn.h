// Host interface between the attention entry (kv8_attn.cu) and the
// prompt-chunk kernel (kv8_chunk.cu).
#pragma once

#include "kv8.cuh"
#include "tc_common.cuh"

namespace w4 {
namespace kv8 {

// Query rows on a key head from which a call takes the prompt-chunk kernel.
// Measured, row tiles of 8 or 16 in the token kernel against tiles of 128, on 2
// sequences of up to 8k keys / 16 of up to 1k, 8 heads (4 of 256 channels), us:
//    64 channels: 96 rows 38 and 43 / 42 and 45, 112 rows 41 and 43 / 45 and 45,
//                 128 rows 44 and 44 / 50 and 45
//   128 channels: 64 rows 45 and 58 / 50 and 57, 80 rows 53 and 58 / 61 and 58,
//                 96 rows 60 and 58 / 71 and 58
//   256 channels: 48 rows 41 and 56 / 46 and 44, 64 rows 46 and 57 / 55 and 45,
//                 96 rows 60 and 57 / 71 and 45
constexpr long long chunk_rows(int D) { return D == 256 ? 49 : D == 128 ? 81 : 113; }

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
