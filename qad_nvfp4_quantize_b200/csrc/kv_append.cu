// nvfp4_kv_append: quantize the new tokens' K and V rows into the pages.
//
// Per block of 16 values: s = E4M3(bmax / (Mt*g)) (Mt = 6, or the better of 6
// and 4), codes E2M1(x * RN(1/(g*s))) with the static global scale g of K or V
// -- the arithmetic of nvfp4_quantize with g_in, bit for bit.
//
// Bound by HBM for prompts in mode MAX (2 B read and 9/16 B written per value),
// by the arithmetic of the two candidates in FOUR_OVER_SIX, and by launch latency
// for single tokens. A lane takes one 16-element block at a time (32 B read, 8 B
// of codes written) of a warp's consecutive tokens, the next one's loads in
// flight meanwhile; the sequence is looked up once and then followed. Measured, 8
// KV heads of 128, single calls on a cold cache: 30,305 tokens (159 MB) in MAX 43
// us (3.7 TB/s), in FOUR_OVER_SIX 63 us (59 back to back); 64 single tokens 8 us.
#include <type_traits>

#include "kernels.h"
#include "kv_common.cuh"

namespace nvfp4 {

constexpr int kAppendWarps = 4;

// kTable: the CTA looks up the steps g*s and their reciprocals (128 scale codes,
// the same values) instead of dividing for each block and candidate.
template <int D, bool kFos, bool kTable>
__global__ void __launch_bounds__(kAppendWarps * 32) kv_append_kernel(
    const uint4* __restrict__ k, const uint4* __restrict__ v, int64_t stride8, KvIndex ix, uint8_t* pages,
    const float* __restrict__ k_g, const float* __restrict__ v_g, int64_t per_warp, int* status) {
  if (blockIdx.x == gridDim.x - 1) {  // reports what is malformed, also where no row leads to it
    for (int b = threadIdx.x; b < ix.batch; b += kAppendWarps * 32) kv_sequence(ix, b, status);
    return;
  }
  const int lane = threadIdx.x & 31;
  const bool is_v = blockIdx.x & 1;
  if (kTable) build_step_table(is_v ? *v_g : *k_g);
  int64_t t = ((int64_t)(blockIdx.x >> 1) * kAppendWarps + (threadIdx.x >> 5)) * per_warp;
  const int64_t last = ix.cu[ix.batch];
  const int64_t rows = last < ix.total ? last : ix.total;  // rows behind the last sequence stay out
  const int64_t t1 = t + per_warp < rows ? t + per_warp : rows;
  constexpr int kBlocks = D / 16;
  const int nblk = ix.hkv * kBlocks;
  int n = lane;  // this lane's block of token t
  auto settle = [&](int64_t& t, int& n) {
    while (n >= nblk) {
      n -= nblk;
      ++t;
    }
  };
  settle(t, n);
  if (t >= t1) return;
  const uint4* x = is_v ? v : k;
  const float g = is_v ? *v_g : *k_g;
  const int gshift = ix.gshift, pshift = gshift + 4;  // log2 of a page's granules and tokens
  Raw16 next;
  load_raw16(x, t * stride8 + 2 * n, NVFP4_IN_BOUNDS(2 * n + 1, stride8, status), next);
  int lo = 0, hi = ix.batch - 1;  // first b with cu[b+1] > t
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if ((int64_t)ix.cu[mid + 1] > t) hi = mid; else lo = mid + 1;
  }
  int b = lo;
  KvSeq seq = kv_sequence(ix, b, nullptr);
  int64_t placed = -1;      // token that `base` belongs to
  uint8_t* base = nullptr;  // its K or V rows of head 0, null where it has no place
  while (t < t1) {
    const Raw16 raw = next;
    const int64_t t0 = t;
    const int n0 = n;
    n += 32;
    settle(t, n);
    if (t < t1) load_raw16(x, t * stride8 + 2 * n, NVFP4_IN_BOUNDS(2 * n + 1, stride8, status), next);
    if (t0 != placed) {
      placed = t0;
      while (b + 1 < ix.batch && t0 >= (int64_t)ix.cu[b + 1]) seq = kv_sequence(ix, ++b, nullptr);
      const int64_t i = t0 - seq.row0, pos = (int64_t)seq.len - seq.rows + i;
      // (rows before cu[0] belong to nobody; a sequence longer than its
      // cache has no such position)
      const bool owned = i >= 0 && i < seq.rows;
      int64_t page = !owned || pos < 0 ? -1 : ix.table[(int64_t)b * ix.width + (pos >> pshift)];
      if (page >= ix.num_pages) page = -1;
      if (owned && page < 0) record_status(status, NVFP4_ERR_PAGE);
      const int slot = (int)pos & (ix.page - 1), row = slot % kGranule;
      base = page < 0 ? nullptr
                      : pages + ((page * ix.hkv << gshift) + slot / kGranule) * granule_bytes(D) + (is_v ? 9 * D : 0) +
                            row * (D / 2);
    }
    if (base == nullptr) continue;
    const float bmax = block_absmax(raw);
    Block q;
    f32x2 xs[8];
    unpack_block(raw, xs);
    if (!isfinite(bmax)) {
      record_status(status, NVFP4_ERR_NONFINITE_INPUT);
      q.sc = 1u;  // the smallest scale and zero codes: the cache holds finite values only
      q.q0 = q.q1 = 0u;
    } else {
      if (kTable)
        quantize_block_tab<false, kFos, false>(xs, bmax, q);
      else
        quantize_block<false, kFos>(xs, bmax, g, 6.0f, q);
      if (kFos) {
        Block q4;
        if (kTable)
          quantize_block_tab<false, true, true>(xs, bmax, q4);
        else
          quantize_block<false, true>(xs, bmax, g, 4.0f, q4);
        if (q4.err < q.err) q = q4;
      }
    }
    const int h = n0 / kBlocks, blk = n0 % kBlocks;
    uint8_t* to = base + ((int64_t)h << gshift) * granule_bytes(D);
    if (!NVFP4_IN_BOUNDS(to + D / 2 - pages, (ix.num_pages * ix.hkv << gshift) * granule_bytes(D), status)) continue;
    *reinterpret_cast<uint2*>(to + blk * 8) = make_uint2(q.q0, q.q1);
    // the scales lie 8*D behind the codes' start; from this row's codes that is 8*D - row*(D/2) + row*(D/16)
    const int row = (int)((seq.len - seq.rows + (t0 - seq.row0)) & (kGranule - 1));
    to[8 * D - row * (D / 2 - D / 16) + blk] = (uint8_t)q.sc;
  }
}

cudaError_t launch_kv_append(const void* k, const void* v, int64_t stride, int D, const KvIndex& ix, uint8_t* pages,
                             const float* k_g, const float* v_g, bool fos, int* status, int num_sms, cudaStream_t s) {
  if (ix.total == 0 || ix.batch == 0) return cudaSuccess;
  // a warp takes consecutive tokens; even CTAs quantize K, odd ones V, the last one checks the offsets and lengths
  const int64_t slots = (int64_t)num_sms * 32;
  const int64_t per_warp = (ix.total + slots - 1) / slots;
  const int64_t warps = (ix.total + per_warp - 1) / per_warp;
  const int grid = 2 * (int)((warps + kAppendWarps - 1) / kAppendWarps) + 1;
  // The table pays for itself where a warp quantizes several tokens twice: in FOUR_OVER_SIX, 8 KV heads of 128, 1 token
  // a warp takes 16.4 us without and 18.4 with it, 2 25.5 and 26.6, 4 42.0 and 41.0, 6 58.4 and 57.4; in MAX, 6 take
  // 38.9 and 40.0.
  const bool table = fos && per_warp >= 4;
  auto pick = [&](auto dim) {
    constexpr int kD = decltype(dim)::value;
    return table ? kv_append_kernel<kD, true, true> : fos ? kv_append_kernel<kD, true, false> : kv_append_kernel<kD, false, false>;
  };
  auto kern = D == 128 ? pick(std::integral_constant<int, 128>{}) : pick(std::integral_constant<int, 64>{});
  note_launch();
  kern<<<grid, kAppendWarps * 32, 0, s>>>(static_cast<const uint4*>(k), static_cast<const uint4*>(v), stride / 8, ix,
                                          pages, k_g, v_g, per_warp, status);
  return cudaGetLastError();
}

}  // namespace nvfp4
