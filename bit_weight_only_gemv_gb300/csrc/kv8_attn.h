// Host interface between the attention entry (kv8_attn.cu) and the
// prompt-chunk kernel (kv8_chunk.cu).
#pragma once

#include "kv8.cuh"
#include "tc_common.cuh"

namespace w4 {
namespace kv8 {

// Query rows on a key head from which a call takes the prompt-chunk kernel.
constexpr int kChunkRows = 17;

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
  CUtensorMap tm_k;
  Cache c;
  Batch bt;
  const __nv_bfloat16* q;
  long long q_stride;
  const float* lse;
  int Hq, G;
  float scale;
  int window;
  int32_t* status;
};

// w4_kv8_weigh for many query rows on a key head (kv8_weigh_tc.cu).
w4_status weigh_many(const WeighParams& p, int dev, w4_stream_t stream);

size_t chunk_workspace_bytes(const Cache& c, const Batch& b, int G, int sms);
w4_status chunk_attn(const Cache& c, const Batch& b, const ChunkArgs& a, void* workspace,
                     int sms, int dev, w4_stream_t stream);

}  // namespace kv8
}  // namespace w4
