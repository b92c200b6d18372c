// nvfp4_kv_append: quantize the new tokens' K and V rows into the pages.
//
// Per block of 16 values: s = E4M3(bmax / (Mt*g)) (Mt = 6, or the better of 6
// and 4), codes E2M1(x * RN(1/(g*s))) with the static global scale g of K or V
// -- the arithmetic of nvfp4_quantize with g_in, bit for bit.
//
// Bound by HBM for prompts (2 B read and 9/16 B written per value) and by
// launch latency for single tokens. One warp takes the K or the V row of one
// token at a time (lane = one 16-element block, 32 B read, 8 B of codes
// written); a warp's tokens are consecutive, so the sequence is looked up once
// and then followed.
#include "kernels.h"
#include "kv_common.cuh"

namespace nvfp4 {

constexpr int kAppendWarps = 4;

template <int D, bool kFos>
__global__ void __launch_bounds__(kAppendWarps * 32) kv_append_kernel(
    const uint4* __restrict__ k, const uint4* __restrict__ v, int64_t stride8, KvIndex ix, uint8_t* pages,
    const float* __restrict__ k_g, const float* __restrict__ v_g, int64_t per_warp, int* status) {
  const int lane = threadIdx.x & 31;
  const int64_t warp = (int64_t)blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
  const bool is_v = warp & 1;
  int64_t t = (warp >> 1) * per_warp;
  const int64_t last = ix.cu[ix.batch];
  const int64_t rows = last < ix.total ? last : ix.total;  // rows behind the last sequence stay out
  const int64_t t1 = t + per_warp < rows ? t + per_warp : rows;
  if (t >= t1) return;
  const uint4* x = is_v ? v : k;
  const float g = is_v ? *v_g : *k_g;
  constexpr int kBlocks = D / 16;
  const int nblk = ix.hkv * kBlocks;
  const int gpp = ix.page / kGranule;
  int lo = 0, hi = ix.batch - 1;  // first b with cu[b+1] > t
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if ((int64_t)ix.cu[mid + 1] > t) hi = mid; else lo = mid + 1;
  }
  int b = lo;
  KvSeq seq = kv_sequence(ix, b, status);
  for (; t < t1; ++t) {
    while (b + 1 < ix.batch && t >= (int64_t)ix.cu[b + 1]) seq = kv_sequence(ix, ++b, status);
    const int64_t i = t - seq.row0;
    const int64_t pos = (int64_t)seq.len - seq.rows + i;
    if (i < 0 || i >= seq.rows || pos < 0) {  // a sequence longer than its cache: no such position
      record_status(status, NVFP4_ERR_PAGE);
      continue;
    }
    const int64_t page = ix.table[(int64_t)b * ix.width + pos / ix.page];
    if (page < 0 || page >= ix.num_pages) {
      record_status(status, NVFP4_ERR_PAGE);
      continue;
    }
    const int slot = (int)(pos % ix.page), row = slot % kGranule;
    uint8_t* base = pages + ((page * ix.hkv) * gpp + slot / kGranule) * granule_bytes(D) + (is_v ? 9 * D : 0);
    for (int n = lane; n < nblk; n += 32) {
      Raw16 raw;
      load_raw16(x, t * stride8 + 2 * n, NVFP4_IN_BOUNDS(2 * n + 1, stride8, status), raw);
      const float bmax = block_absmax(raw);
      Block q;
      f32x2 xs[8];
      unpack_block(raw, xs);
      if (!isfinite(bmax)) {
        record_status(status, NVFP4_ERR_NONFINITE_INPUT);
        q.sc = 1u;  // the smallest scale and zero codes: the cache holds finite values only
        q.q0 = q.q1 = 0u;
      } else {
        quantize_block<false, kFos>(xs, bmax, g, 6.0f, q);
        if (kFos) {
          Block q4;
          quantize_block<false, true>(xs, bmax, g, 4.0f, q4);
          if (q4.err < q.err) q = q4;
        }
      }
      const int h = n / kBlocks, blk = n % kBlocks;
      uint8_t* gr = base + (int64_t)h * gpp * granule_bytes(D);
      if (!NVFP4_IN_BOUNDS(gr + 9 * D - pages, ix.num_pages * ix.hkv * gpp * granule_bytes(D) + 1, status)) continue;
      *reinterpret_cast<uint2*>(gr + row * (D / 2) + blk * 8) = make_uint2(q.q0, q.q1);
      gr[8 * D + row * kBlocks + blk] = (uint8_t)q.sc;
    }
  }
}

cudaError_t launch_kv_append(const void* k, const void* v, int64_t stride, int D, const KvIndex& ix, uint8_t* pages,
                             const float* k_g, const float* v_g, bool fos, int* status, int num_sms, cudaStream_t s) {
  if (ix.total == 0 || ix.batch == 0) return cudaSuccess;
  // two warps (K, V) per group of consecutive tokens; at most 16 warps per scheduler slot of the card
  const int64_t slots = (int64_t)num_sms * 32;
  const int64_t per_warp = (ix.total + slots - 1) / slots;
  const int64_t warps = 2 * ((ix.total + per_warp - 1) / per_warp);
  const int grid = (int)((warps + kAppendWarps - 1) / kAppendWarps);
  auto kern = D == 128 ? (fos ? kv_append_kernel<128, true> : kv_append_kernel<128, false>)
                       : (fos ? kv_append_kernel<64, true> : kv_append_kernel<64, false>);
  note_launch();
  kern<<<grid, kAppendWarps * 32, 0, s>>>(static_cast<const uint4*>(k), static_cast<const uint4*>(v), stride / 8, ix,
                                          pages, k_g, v_g, per_warp, status);
  return cudaGetLastError();
}

}  // namespace nvfp4
