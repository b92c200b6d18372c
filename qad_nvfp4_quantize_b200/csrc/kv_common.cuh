// Layout and index arithmetic of the paged NVFP4 KV cache (kv_append.cu,
// kv_pages.cu, kv_attention.cu, kv_prefill.cu). The storage follows "Developing Nemotron 3.5
// Lightning NVFP4 with QAD using NVIDIA Model Optimizer", Table 1
// "four_over_six + NVFP4 KV": K and V in NVFP4 (blocks of 16 along the head
// dimension, one static FP32 global scale each), attention in 16-bit floating
// point on the dequantized values.
//
// Granule: 16 consecutive tokens of one KV head, 18*D bytes, contiguous:
//   K codes [16][D/2] | K scales [16][D/16] | V codes [16][D/2] | V scales
// A page holds page_size/16 granules per head: pages [P][Hkv][page/16][18*D].
// One bulk copy therefore fetches all that attention needs of 16 tokens, for
// every page size, and a page is one contiguous piece for the copies.
#pragma once

#include "block_math.cuh"

namespace nvfp4 {

constexpr int kGranule = 16;  // tokens

__host__ __device__ constexpr int granule_bytes(int D) { return 18 * D; }

// What every KV kernel needs to find a token: sequence b owns rows
// [cu[b], cu[b+1]) of the new tokens; its token i sits at position
// kv_len[b] - (cu[b+1] - cu[b]) + i; page j of the sequence is table[b*width+j].
struct KvIndex {
  const int32_t* cu;
  const int32_t* kv_len;
  const int32_t* table;
  int batch, width, page, hkv;
  int64_t total;      // rows of the new-token tensors
  int64_t num_pages;
  int gshift;         // log2 of the granules in a page
};

// Rows and cached length of a sequence, brought into the tensors' extents. A
// malformed offset or length (negative, decreasing, beyond the rows or the
// table) is recorded and cut off, so that no access leaves a buffer.
struct KvSeq {
  int64_t row0;
  int32_t rows, len;
};
NVFP4_DEVINL KvSeq kv_sequence(const KvIndex& ix, int b, int* status) {
  const int64_t a = ix.cu[b], e = ix.cu[b + 1];
  const int64_t len = ix.kv_len[b], most = (int64_t)ix.width * ix.page;
  KvSeq s;
  s.row0 = a;
  const bool ok = a >= 0 && a <= e && e <= ix.total;
  s.rows = ok ? (int32_t)(e - a) : 0;
  s.len = (int32_t)(len < 0 ? 0 : len > most ? most : len);
  if (!ok || len < 0 || len > most) record_status(status, NVFP4_ERR_PAGE);
  return s;
}

}  // namespace nvfp4
