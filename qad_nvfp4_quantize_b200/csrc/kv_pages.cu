// Page management of the paged NVFP4 KV cache: copy, fork, free and compact.
// The pool's state is refs[P] (sequences that hold a page; 0 = free),
// block_table[S][W] and seq_len[S] (tokens held by a slot). Everything stays
// on the device; results do not depend on thread order (pages are taken and
// moved in ascending index order, counts are integer sums).
#include "kernels.h"
#include "kv_common.cuh"

namespace nvfp4 {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;

// Block-wide exclusive scan of one int per thread; *total gets the sum.
// `sh` holds kPlanWarps + 1 ints.
__device__ __forceinline__ int block_exclusive_scan(int v, int* sh, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += u;
  }
  __syncthreads();  // the last scan's readers are done with sh
  if (lane == 31) sh[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    const int nw = blockDim.x >> 5;
    int w = lane < nw ? sh[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xFFFFFFFFu, w, o);
      if (lane >= o) w += u;
    }
    if (lane < nw) sh[lane] = w;
    if (lane == nw - 1) sh[kPlanWarps] = w;
  }
  __syncthreads();
  *total = sh[kPlanWarps];
  return incl - v + (warp > 0 ? sh[warp - 1] : 0);
}

// ------------------------------------------------------------------ copying
// Page src[i] -> page dst[i]; entries with a negative index are skipped. Bound
// by HBM (each byte read and written once). A CTA copies pieces of 32 KB, eight
// 16-byte loads in flight per thread (compacting 16,384 pages of 74 KB: 110 to
// 112 us for the whole call on a cold cache, 107 back to back; with four loads 120
// where this took 111); an entry is as many pieces as its page
// needs, so a few large pages spread over the card too. Where a page is copied
// many times the writes bound it: 151 MB take 43 us, as filling that much does.
constexpr int kRowThreads = 256;
constexpr int kCopyThreads = 256, kCopyLoads = 8;
constexpr int kCopyPiece = kCopyThreads * kCopyLoads;  // 16-byte vectors

__global__ void __launch_bounds__(kCopyThreads) kv_copy_kernel(uint4* pages, int64_t num_pages, int64_t page_vecs,
                                                               const int32_t* __restrict__ src,
                                                               const int32_t* __restrict__ dst, int pieces,
                                                               int64_t units, int* status) {
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int64_t i = u / pieces;
    const int64_t a = src[i], b = dst[i];
    if (a < 0 || b < 0) continue;
    if (a >= num_pages || b >= num_pages) {
      record_status(status, NVFP4_ERR_PAGE);
      continue;
    }
    const int64_t at = (u - i * pieces) * kCopyPiece + threadIdx.x;
    const uint4* from = pages + a * page_vecs;
    uint4* to = pages + b * page_vecs;
    uint4 r[kCopyLoads];
#pragma unroll
    for (int e = 0; e < kCopyLoads; ++e)
      if (at + e * kCopyThreads < page_vecs &&
          NVFP4_IN_BOUNDS(a * page_vecs + at + e * kCopyThreads, num_pages * page_vecs, status))
        r[e] = ld_stream(from + at + e * kCopyThreads);
#pragma unroll
    for (int e = 0; e < kCopyLoads; ++e)
      if (at + e * kCopyThreads < page_vecs &&
          NVFP4_IN_BOUNDS(b * page_vecs + at + e * kCopyThreads, num_pages * page_vecs, status))
        to[at + e * kCopyThreads] = r[e];
  }
}

cudaError_t launch_kv_copy(uint8_t* pages, int64_t num_pages, int64_t page_bytes, const int32_t* src,
                           const int32_t* dst, int64_t n, int* status, int num_sms, cudaStream_t s) {
  if (n == 0) return cudaSuccess;
  const int64_t vecs = page_bytes / 16;
  const int pieces = (int)((vecs + kCopyPiece - 1) / kCopyPiece);
  const int64_t units = n * pieces, most = (int64_t)num_sms * 8;
  note_launch();
  kv_copy_kernel<<<(int)(units < most ? units : most), kCopyThreads, 0, s>>>(
      reinterpret_cast<uint4*>(pages), num_pages, vecs, src, dst, pieces, units, status);
  return cudaGetLastError();
}

// ------------------------------------------------------------------ forking
struct PoolIndex {
  int32_t* refs;
  int32_t* table;
  int32_t* seq_len;
  int64_t num_pages;
  int slots, width, page;
};

// Tokens of a slot, cut to what its row of the table can hold.
NVFP4_DEVINL int32_t slot_len(const PoolIndex& p, int32_t slot, int* status) {
  const int64_t len = p.seq_len[slot], most = (int64_t)p.width * p.page;
  if (len < 0 || len > most) record_status(status, NVFP4_ERR_PAGE);
  return (int32_t)(len < 0 ? 0 : len > most ? most : len);
}

// Entry j of child i's row of the table: a shared page counted once more, or the
// part page's copy.
NVFP4_DEVINL void fork_entry(const PoolIndex& p, int a, int c, int to, int64_t j, int* status) {
  const int64_t full = p.seq_len[c] / p.page;
  if (j > full || (j == full && to < 0)) return;
  if (!NVFP4_IN_BOUNDS(j, p.width, status) || !NVFP4_IN_BOUNDS(a, p.slots, status) ||
      !NVFP4_IN_BOUNDS(c, p.slots, status))
    return;
  if (j < full) {
    const int64_t page = p.table[(int64_t)a * p.width + j];
    p.table[(int64_t)c * p.width + j] = (int32_t)page;
    if (page < 0 || page >= p.num_pages)
      record_status(status, NVFP4_ERR_PAGE);
    else
      atomicAdd(&p.refs[page], 1);
  } else {
    p.table[(int64_t)c * p.width + j] = to;
  }
}

// One CTA: which entries are sound, which pages the part pages are copied to.
// src[i], dst[i] = the part page and its copy, -1 where the parent ends with a
// full page, -2 where the entry is refused (a slot out of range, a child that
// holds tokens or is named by an earlier entry, parent == child). Bound by
// latency: a handful of block-wide scans; the search for free pages walks the
// reference counts 16 to a thread and stops at the last one needed.
__global__ void __launch_bounds__(kPlanThreads) kv_fork_plan_kernel(PoolIndex p, const int32_t* __restrict__ parent,
                                                                    const int32_t* __restrict__ child, int n,
                                                                    int32_t* src, int32_t* dst, int with_rows,
                                                                    int* status) {
  __shared__ int sh[kPlanWarps + 1];
  const int t = threadIdx.x;
  // dst[i] holds the parent's length until its page is known
  for (int i = t; i < n; i += kPlanThreads) {
    const int a = parent[i], c = child[i];
    bool ok = a >= 0 && a < p.slots && c >= 0 && c < p.slots && a != c;
    if (ok) ok = p.seq_len[c] == 0;
    src[i] = ok ? -1 : -2;
    dst[i] = ok ? slot_len(p, a, status) : 0;
    if (!ok) record_status(status, NVFP4_ERR_PAGE);
  }
  __syncthreads();
  // the first entry that names a child has it: the lowest of the claims i - n < 0
  for (int i = t; i < n; i += kPlanThreads)
    if (src[i] == -1) atomicMin(&p.seq_len[child[i]], i - n);
  __syncthreads();
  for (int i = t; i < n; i += kPlanThreads)
    if (src[i] == -1 && *(volatile int32_t*)&p.seq_len[child[i]] != i - n) {
      src[i] = -2;
      record_status(status, NVFP4_ERR_PAGE);
    }
  __syncthreads();
  // each child's length; the rank of its part page among all of them (kept in src)
  int need = 0;
  for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
    const int i = i0 + t;
    const bool ok = i < n && src[i] == -1;
    const int len = ok ? dst[i] : 0;
    const int part = len % p.page ? 1 : 0;
    int sum;
    const int rank = need + block_exclusive_scan(part, sh, &sum);
    need += sum;
    if (ok) {
      p.seq_len[child[i]] = len;
      if (part) src[i] = rank;
    }
  }
  __syncthreads();
  // dst[r] = the r-th free page
  int found = 0;
  for (int64_t p0 = 0; p0 < p.num_pages && found < need; p0 += 16 * kPlanThreads) {
    const int64_t at = p0 + 16 * t;
    uint32_t mask = 0;
    if (at + 16 <= p.num_pages && (reinterpret_cast<uintptr_t>(p.refs) & 15u) == 0) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int4 r = *reinterpret_cast<const int4*>(p.refs + at + 4 * e);
        mask |= (uint32_t)((r.x == 0) | (r.y == 0) << 1 | (r.z == 0) << 2 | (r.w == 0) << 3) << (4 * e);
      }
    } else {
      for (int e = 0; e < 16; ++e)
        if (at + e < p.num_pages && p.refs[at + e] == 0) mask |= 1u << e;
    }
    int sum;
    int r = found + block_exclusive_scan(__popc(mask), sh, &sum);
    found += sum;
    for (; mask && r < need; mask &= mask - 1, ++r)
      if (NVFP4_IN_BOUNDS(r, n, status) && NVFP4_IN_BOUNDS(at + __ffs(mask) - 1, p.num_pages, status))
        dst[r] = (int32_t)(at + __ffs(mask) - 1);
  }
  __syncthreads();
  if (found < need) {  // too few: the pool stays as it was
    for (int i = t; i < n; i += kPlanThreads) {
      if (src[i] != -2) p.seq_len[child[i]] = 0;
      src[i] = -2;
      dst[i] = -2;
    }
    if (t == 0) record_status(status, NVFP4_ERR_NO_PAGES);
    return;
  }
  // entry i takes dst[rank], rank <= i: the highest entries first, so that no rank is overwritten before it is read
  for (int i0 = (n - 1) / kPlanThreads * kPlanThreads; i0 >= 0; i0 -= kPlanThreads) {
    const int i = i0 + t;
    const int r = i < n ? src[i] : -2;
    const int page = r >= 0 && NVFP4_IN_BOUNDS(r, n, status) ? dst[r] : r;
    __syncthreads();
    if (i < n) {
      dst[i] = page;
      if (r >= 0) {
        const int a = parent[i];
        const int64_t from = (int64_t)a * p.width + p.seq_len[child[i]] / p.page;
        const int64_t part = NVFP4_IN_BOUNDS(from, (int64_t)p.slots * p.width, status) ? p.table[from] : -1;
        if (NVFP4_IN_BOUNDS(page, p.num_pages, status)) p.refs[page] = 1;
        if (part < 0 || part >= p.num_pages) record_status(status, NVFP4_ERR_PAGE);
        src[i] = part < 0 || part >= p.num_pages ? -1 : (int32_t)part;  // nothing to copy from
      }
    }
    __syncthreads();
  }
  if (!with_rows) return;
  for (int64_t e = t; e < (int64_t)n * p.width; e += kPlanThreads) {
    const int i = (int)(e / p.width);
    if (dst[i] != -2) fork_entry(p, parent[i], child[i], dst[i], e - (int64_t)i * p.width, status);
  }
}

// A small fork's rows are written by the planning CTA itself: one launch less
// (3 us of host time, 2 us on the device) for up to this many entries.
constexpr int64_t kForkRowsInPlan = 4 * kPlanThreads;

// The children's rows of the table, a CTA for each 256 entries. Bound by the
// atomics' latency.
__global__ void __launch_bounds__(kRowThreads) kv_fork_rows_kernel(PoolIndex p, const int32_t* __restrict__ parent,
                                                                   const int32_t* __restrict__ child,
                                                                   const int32_t* __restrict__ dst, int* status) {
  const int i = blockIdx.x, to = dst[i];
  if (to == -2) return;
  fork_entry(p, parent[i], child[i], to, (int64_t)blockIdx.y * kRowThreads + threadIdx.x, status);
}

cudaError_t launch_kv_fork(const PoolArgs& a, const int32_t* parent, const int32_t* child, int n, int32_t* src,
                           int32_t* dst, int* status, cudaStream_t s) {
  if (n == 0) return cudaSuccess;
  const PoolIndex p{a.refs, a.table, a.seq_len, a.num_pages, a.slots, a.width, a.page};
  note_launch();
  const bool with_rows = (int64_t)n * a.width <= kForkRowsInPlan;
  kv_fork_plan_kernel<<<1, kPlanThreads, 0, s>>>(p, parent, child, n, src, dst, with_rows, status);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || with_rows) return e;
  note_launch();
  const dim3 grid((unsigned)n, (unsigned)((a.width + kRowThreads - 1) / kRowThreads));
  kv_fork_rows_kernel<<<grid, kRowThreads, 0, s>>>(p, parent, child, dst, status);
  return cudaGetLastError();
}

// ------------------------------------------------------------------ freeing
// One CTA a named slot. The exchange of the slot's length gives its pages to
// the first CTA that comes: a slot that is named twice is freed once.
__global__ void __launch_bounds__(kRowThreads) kv_free_kernel(PoolIndex p, const int32_t* __restrict__ which,
                                                              int* status) {
  __shared__ int64_t held;
  const int slot = which[blockIdx.x];
  if (threadIdx.x == 0) {
    held = 0;
    if (slot < 0 || slot >= p.slots) {
      record_status(status, NVFP4_ERR_PAGE);
    } else {
      const int64_t len = atomicExch(&p.seq_len[slot], 0), most = (int64_t)p.width * p.page;
      if (len < 0 || len > most) record_status(status, NVFP4_ERR_PAGE);
      held = ((len < 0 ? 0 : len > most ? most : len) + p.page - 1) / p.page;
    }
  }
  __syncthreads();
  for (int64_t j = threadIdx.x; j < held; j += kRowThreads) {
    if (!NVFP4_IN_BOUNDS((int64_t)slot * p.width + j, (int64_t)p.slots * p.width, status)) continue;
    int32_t* at = p.table + (int64_t)slot * p.width + j;
    const int64_t page = *at;
    *at = -1;
    if (page < 0 || page >= p.num_pages) {
      record_status(status, NVFP4_ERR_PAGE);
    } else if (atomicSub(&p.refs[page], 1) <= 0) {  // nobody held it
      atomicAdd(&p.refs[page], 1);
      record_status(status, NVFP4_ERR_PAGE);
    }
  }
}

cudaError_t launch_kv_free(const PoolArgs& a, const int32_t* which, int n, int* status, cudaStream_t s) {
  if (n == 0) return cudaSuccess;
  note_launch();
  kv_free_kernel<<<n, kRowThreads, 0, s>>>(PoolIndex{a.refs, a.table, a.seq_len, a.num_pages, a.slots, a.width, a.page},
                                           which, status);
  return cudaGetLastError();
}

// --------------------------------------------------------------- compacting
// L = used pages. The i-th used page at or above L moves to the i-th free page
// below L (there are as many of one as of the other). Launches: the used pages of
// each chunk of 4096 (up to 8 chunks are counted in the next one instead: 3 us of
// host time and a launch less, against reading them all); ranks, moves
// and reference counts; the tables and the moved pages' counts.
constexpr int kChunkPages = 4 * kPlanThreads, kSmallChunks = 8;

NVFP4_DEVINL uint32_t used_mask(const int32_t* refs, int64_t at, int64_t n) {
  uint32_t m = 0;
  if (at + 4 <= n && (reinterpret_cast<uintptr_t>(refs) & 15u) == 0) {  // at is a multiple of 4
    const int4 r = *reinterpret_cast<const int4*>(refs + at);
    return (uint32_t)((r.x > 0) | (r.y > 0) << 1 | (r.z > 0) << 2 | (r.w > 0) << 3);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (at + e < n && refs[at + e] > 0) m |= 1u << e;
  return m;
}

__global__ void __launch_bounds__(kPlanThreads) kv_compact_count_kernel(const int32_t* __restrict__ refs, int64_t n,
                                                                        int32_t* counts) {
  __shared__ int sh[kPlanWarps + 1];
  int sum;
  block_exclusive_scan(__popc(used_mask(refs, (int64_t)blockIdx.x * kChunkPages + 4 * threadIdx.x, n)), sh, &sum);
  if (threadIdx.x == 0) counts[blockIdx.x] = sum;
}

__global__ void __launch_bounds__(kPlanThreads) kv_compact_plan_kernel(const int32_t* refs, int64_t n,
                                                                       const int32_t* counted, int chunks,
                                                                       int32_t* refs_out, int32_t* src, int32_t* dst,
                                                                       int64_t cap, int32_t* rank_of, int32_t* live,
                                                                       int* status) {
  __shared__ int sh[kPlanWarps + 1];
  __shared__ int32_t small[kSmallChunks];
  const int t = threadIdx.x;
  const int32_t* counts = counted;
  if (counted == nullptr) {  // at most kSmallChunks, all loads in flight
    uint32_t used[kSmallChunks];
#pragma unroll
    for (int c = 0; c < kSmallChunks; ++c) used[c] = used_mask(refs, (int64_t)c * kChunkPages + 4 * t, n);
    if (t < kSmallChunks) small[t] = 0;
    __syncthreads();
#pragma unroll
    for (int c = 0; c < kSmallChunks; ++c) {
      const int sum = __reduce_add_sync(0xFFFFFFFFu, __popc(used[c]));
      if ((t & 31) == 0) atomicAdd(&small[c], sum);
    }
    __syncthreads();
    counts = small;
  }
  int total = 0, before = 0;  // used pages in all, and in the chunks before this one
  for (int c0 = 0; c0 < chunks; c0 += kPlanThreads) {
    const int c = c0 + t;
    const int v = c < chunks ? counts[c] : 0;
    int sum;
    block_exclusive_scan(v, sh, &sum);
    total += sum;
    block_exclusive_scan(c < (int)blockIdx.x ? v : 0, sh, &sum);
    before += sum;
  }
  const int64_t L = total;
  // used pages below L: the whole chunks before L's, then a part of that one
  const int lc = (int)(L / kChunkPages);
  int below = 0;
  for (int c0 = 0; c0 < lc; c0 += kPlanThreads) {
    const int c = c0 + t;
    int sum;
    block_exclusive_scan(c < lc ? counts[c] : 0, sh, &sum);
    below += sum;
  }
  {
    int sum;
    block_exclusive_scan(__popc(used_mask(refs, (int64_t)lc * kChunkPages + 4 * t, L)), sh, &sum);
    below += sum;
  }
  const int moves = total - below;
  const int64_t at = (int64_t)blockIdx.x * kChunkPages + 4 * t;
  const uint32_t used = used_mask(refs, at, n);
  int sum;
  int rank = before + block_exclusive_scan(__popc(used), sh, &sum);  // used pages before this one
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int64_t p = at + e;
    if (p >= n) break;
    const bool u = (used >> e) & 1u;
    if (p < L) {
      if (u) refs_out[p] = refs[p];
      else if (NVFP4_IN_BOUNDS(p - rank, cap, status)) dst[p - rank] = (int32_t)p;  // (its count comes with its new page)
    } else if (u) {
      if (NVFP4_IN_BOUNDS(rank - below, cap, status)) src[rank - below] = (int32_t)p;
      rank_of[p] = rank - below;
    } else {
      refs_out[p] = 0;
      rank_of[p] = -1;
    }
    rank += u;
  }
  for (int64_t r = (int64_t)blockIdx.x * kPlanThreads + t; r < cap; r += (int64_t)gridDim.x * kPlanThreads)
    if (r >= moves) src[r] = dst[r] = -1;
  if (blockIdx.x == 0 && t == 0) *live = total;
}

// The first ref_blocks CTAs: the moved pages' reference counts; the others: 256
// entries of a row of the table each. In place or not: the rows read no counts.
__global__ void __launch_bounds__(kRowThreads) kv_compact_apply_kernel(PoolIndex p, const int32_t* __restrict__ src,
                                                                       const int32_t* __restrict__ dst, int64_t cap,
                                                                       const int32_t* __restrict__ rank_of,
                                                                       const int32_t* __restrict__ live,
                                                                       int32_t* refs_out, int32_t* table_out,
                                                                       int ref_blocks, int* status) {
  if ((int)blockIdx.x < ref_blocks) {
    for (int64_t r = (int64_t)blockIdx.x * kRowThreads + threadIdx.x; r < cap; r += (int64_t)ref_blocks * kRowThreads) {
      const int32_t a = src[r];
      if (a < 0) return;  // the moves come first
      const int32_t b = dst[r];
      if (!NVFP4_IN_BOUNDS(a, p.num_pages, status) || !NVFP4_IN_BOUNDS(b, p.num_pages, status)) continue;
      const int32_t count = p.refs[a];
      refs_out[b] = count;
      refs_out[a] = 0;
    }
    return;
  }
  const int64_t L = *live, pieces = (p.width + kRowThreads - 1) / kRowThreads;
  for (int64_t x = blockIdx.x - ref_blocks; x < p.slots * pieces; x += gridDim.x - ref_blocks) {
    const int64_t row = x / pieces, j = (x - row * pieces) * kRowThreads + threadIdx.x;
    if (j >= p.width) continue;
    const int64_t held = (slot_len(p, (int32_t)row, status) + (int64_t)p.page - 1) / p.page;
    int64_t page = p.table[row * p.width + j];
    if (j < held) {
      if (page < 0 || page >= p.num_pages || (page >= L && rank_of[page] < 0))
        record_status(status, NVFP4_ERR_PAGE);  // not a page of this pool, or one that nobody holds
      else if (page >= L && NVFP4_IN_BOUNDS(rank_of[page], cap, status))
        page = dst[rank_of[page]];
    }
    if (!NVFP4_IN_BOUNDS(row * p.width + j, (int64_t)p.slots * p.width, status)) continue;
    table_out[row * p.width + j] = (int32_t)page;
  }
}

size_t kv_compact_workspace_bytes(int64_t num_pages) {
  const int64_t chunks = (num_pages + kChunkPages - 1) / kChunkPages;
  return (size_t)(4 * (num_pages + chunks) + 16);
}

cudaError_t launch_kv_compact(const PoolArgs& a, int32_t* refs_out, int32_t* table_out, int32_t* src, int32_t* dst,
                              int32_t* live, void* workspace, int* status, int num_sms, cudaStream_t s) {
  const int64_t n = a.num_pages, cap = n / 2 > 1 ? n / 2 : 1;
  const int chunks = (int)((n + kChunkPages - 1) / kChunkPages);
  int32_t* rank_of = static_cast<int32_t*>(workspace);
  int32_t* counts = rank_of + n;
  const PoolIndex p{a.refs, a.table, a.seq_len, n, a.slots, a.width, a.page};
  cudaError_t e;
  if (chunks > kSmallChunks) {
    note_launch();
    kv_compact_count_kernel<<<chunks, kPlanThreads, 0, s>>>(a.refs, n, counts);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  note_launch();
  kv_compact_plan_kernel<<<chunks, kPlanThreads, 0, s>>>(a.refs, n, chunks > kSmallChunks ? counts : nullptr, chunks,
                                                        refs_out, src, dst, cap, rank_of, live, status);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  note_launch();
  const int64_t refs = (cap + kRowThreads - 1) / kRowThreads, most = 16 * (int64_t)num_sms;
  const int64_t rows = a.slots * ((a.width + (int64_t)kRowThreads - 1) / kRowThreads);
  const int ref_blocks = (int)(refs < num_sms ? refs : num_sms);
  const int row_blocks = (int)(rows < 1 ? 1 : rows < most ? rows : most);
  kv_compact_apply_kernel<<<ref_blocks + row_blocks, kRowThreads, 0, s>>>(p, src, dst, cap, rank_of, live, refs_out,
                                                                         table_out, ref_blocks, status);
  return cudaGetLastError();
}

}  // namespace nvfp4
