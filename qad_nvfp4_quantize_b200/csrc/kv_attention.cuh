// What the two attention kernels over the paged NVFP4 cache share: the
// dequantization to FP16, the masks' limits and the workspace.
//
// Number format. A cached value is g * s * c with s an E4M3 scale and c an E2M1
// code; s*c has at most 6 significant bits. The hardware converts two codes at a
// time to FP16, exactly; the scale's seven bits, placed at FP16's exponent and
// mantissa, read as s * 2^-8 (subnormals included). The kernels multiply the
// two: c*s * 2^-8, a multiple of 2^-18 of at most 6 * 480 * 2^-8 = 11.25, so
// FP16 holds it exactly. The factor 2^8 * g joins the softmax scale (K) and the
// final division (V). Moving the codes' bits instead of converting them cost
// 0.081 cycles per eight codes and SM against 0.023, and was half of the
// instructions of both attention kernels.
// The bits read the E4M3 NaN code 0x7F as 480 and drop the sign, so no cache
// content is infinite or NaN: what a mask hides cannot reach a row's result
// through 0 * NaN.
#pragma once

#include "kernels.h"
#include "kv_common.cuh"

namespace nvfp4 {

NVFP4_DEVINL uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Eight codes of a word -> four FP16 pairs, (0,1) (2,3) (4,5) (6,7).
NVFP4_DEVINL void codes_to_half(uint32_t w, uint32_t (&p)[4]) {
  asm("{\n\t.reg .b8 q0, q1, q2, q3;\n\tmov.b32 {q0, q1, q2, q3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, q0;\n\tcvt.rn.f16x2.e2m1x2 %1, q1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, q2;\n\tcvt.rn.f16x2.e2m1x2 %3, q3;\n\t}"
      : "=r"(p[0]), "=r"(p[1]), "=r"(p[2]), "=r"(p[3])
      : "r"(w));
}

constexpr int kValueExp = 8;            // cached values are held as k, v / g * 2^-8
// What O / l is multiplied by: 2^8 * g, in an order that passes FP32's range only where the output does.
NVFP4_DEVINL float output_factor(float vg, float l) { return 256.0f / l * vg; }

// Two E4M3 scales (low bytes of each half) -> FP16 pair s * 2^-8.
NVFP4_DEVINL uint32_t scales_to_half(uint32_t two) { return (two & 0x007F007Fu) << 7; }

NVFP4_DEVINL float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

NVFP4_DEVINL float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Maxima that are NaN if an argument is.
NVFP4_DEVINL float max2_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
NVFP4_DEVINL float max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Power of two that brings a row of BF16 queries whose largest magnitude is
// amax to [2^14, 2^15), as the exponent to add (0 for a non-finite row; a zero
// or subnormal one gets the largest). FP16 then holds every query exactly down to 2^-29 of the row's largest,
// and to 2^-40 of it below.
NVFP4_DEVINL int query_exponent(float amax) {
  const int e = (int)((__float_as_uint(amax) >> 23) & 0xFFu);
  return e == 255 ? 0 : 14 + 127 - (e > 0 ? e : 1);
}
// x * 2^e for |e| up to 140 (two exact factors; a subnormal x stays one).
NVFP4_DEVINL float scale_exp2(float x, int e) {
  const int h = e / 2;
  return x * __uint_as_float((uint32_t)(127 + h) << 23) * __uint_as_float((uint32_t)(127 + e - h) << 23);
}

// Cached tokens that the new token at position `pos` sees: [lo, hi).
struct Visible {
  int32_t lo, hi;
};
NVFP4_DEVINL Visible visible(int64_t pos, int32_t len, int causal, int64_t window) {
  int64_t hi = causal ? (pos + 1 < len ? pos + 1 : len) : len;
  int64_t lo = window > 0 ? pos - window + 1 : 0;
  if (lo < 0) lo = 0;
  if (hi < lo) hi = lo;
  return Visible{(int32_t)lo, (int32_t)hi};
}

// Division of 0 <= n < 2^31 by a divisor known to the host: with l = ceil(log2 d)
// and m = floor(2^(31+l) / d) + 1, m * d exceeds 2^(31+l) by at most 2^l, which
// no such n notices.
struct Divisor {
  uint32_t d, m;
  int shift;
  Divisor() = default;
  explicit Divisor(uint32_t of) : d(of) {
    int l = 0;
    while ((uint64_t(1) << l) < of) ++l;
    shift = 31 + l;
    m = (uint32_t)((uint64_t(1) << shift) / of + 1);
  }
  NVFP4_DEVINL int32_t divide(int32_t n) const { return (int32_t)(((uint64_t)(uint32_t)n * m) >> shift); }
};

struct AttnArgs {
  const uint16_t* q;   // BF16 [total][hq][D], rows q_stride apart
  int64_t q_stride;
  KvIndex ix;
  const uint8_t* pages;
  const float *k_g, *v_g;
  float scale;         // softmax scale
  int group;           // query heads per KV head
  Divisor by_group, by_grid;
  int causal;
  int64_t window;      // 0: no window; below 2^31
  uint16_t* out;       // BF16 [total][hq][D]
  float* lse;          // FP32 [total][hq] or null
  float* partial;      // workspace
  int32_t* counters;   // workspace, zero between calls
  int* status;
  int64_t wait_cycles;  // bound of every wait
  int withheld;         // 1 in the self-test: the first copies are awaited but not issued
};

// One thread's arrival, after a barrier of its CTA, at a counter of CTAs that
// have stored their parts: true for the last of `others` + 1, which may then
// read all of them (behind another barrier). The counter is zero again.
NVFP4_DEVINL int arrive_last(int32_t* counter, int others) {
  int before;
  asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(before) : "l"(counter) : "memory");
  if (before == others) *counter = 0;
  return before == others;
}

constexpr int64_t kAttnWaitCycles = 4000000000ll;  // about 2 s
// The running maximum m of a row is held kHeadroom below the score that set it (in log2 units) and may lag kRescaleAt
// behind a larger one, so a row's largest weight 2^(s - m) lies in [2^7, 2^15]: weights are FP16 operands, which hold
// 11 bits down to 2^-14 and multiples of 2^-24 below. Without the head-room tokens 16 nats below an attention sink lost
// their weights, and those more than 17.3 below it vanished from the output.
constexpr float kRescaleAt = 8.0f, kHeadroom = 7.0f;
constexpr float kStartMax = -3.40282347e38f;       // running maximum before the first visible token
// A weight is 2^(s * factor - m) by one FMA: the product is not rounded, m is, by half a step of the score. From 2^24 on
// that can lift a weight above FP16, from 2^28 on every largest one. A row whose factor would let its scores (at most D
// products of 2^15 and 11.25) reach 2^22 has them multiplied first, rounded as m is.
template <int D>
constexpr float kHugeFactor = 4194304.0f / (D * 368640.0f);
constexpr float kLog2e = 1.44269504f, kLn2 = 0.693147181f;

// A row whose largest new score is `top` keeps its running maximum m, whatever
// its neighbours do, or takes a new one where top exceeds m by more.
NVFP4_DEVINL bool exceeds(float top, float m) { return top - m > kRescaleAt + kHeadroom; }
NVFP4_DEVINL float new_max(float top, float m) { return exceeds(top, m) ? top - kHeadroom : m; }

// The same value in every lane, in a form that the compiler knows to be uniform.
NVFP4_DEVINL int uniform(int v) { return __reduce_max_sync(0xFFFFFFFFu, v); }

// Wait of a whole warp for a phase of an mbarrier, given up (false) after
// `cycles` or when another warp gave up. Every lane polls: one lane
// polling for the others measured 580 cycles from arrival to return with 16
// warps waiting, this 130.
NVFP4_DEVINL bool wait_bounded(uint64_t* bar, uint32_t parity, volatile int* abort, int64_t cycles) {
  if (__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity))) return true;
  uint32_t spins = 0;
  const int64_t t0 = clock64();
  while (true) {
    const bool done = mbar_try_wait(bar, parity);
    if (__all_sync(0xFFFFFFFFu, done)) return true;
    if ((++spins & 15u) == 0 && __any_sync(0xFFFFFFFFu, *abort || clock64() - t0 > cycles)) {
      *abort = 1;
      return false;
    }
  }
}

// A warp that gave up lets what may be in flight (copies, MMAs) arrive, 1 ms at
// most: it must not land in a CTA that gets the same memory later.
NVFP4_DEVINL void settle(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity) && globaltimer_ns() - t0 < 1000000ull) {
  }
}

// The queries and the page table, asked for while the lengths are on their way:
// what find_part's caller reads next then waits in L2. A line each thread; what
// lies behind the grid's first line each is left out.
NVFP4_DEVINL void prefetch_inputs(const AttnArgs& a, int head_dim) {
  auto ask = [](const void* p, int64_t bytes, int64_t at) {
    if (at < bytes) asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char*>(p) + at));
  };
  const int64_t at = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * 128;
  ask(a.q, ((a.ix.total - 1) * a.q_stride + (int64_t)a.ix.hkv * a.group * head_dim) * 2, at);
  ask(a.ix.table, (int64_t)a.ix.batch * a.ix.width * 4, at);
  ask(a.k_g, 4, at);
  ask(a.v_g, 4, at);
}

// ---------------------------------------------------------------------------
// Work list. A work is one KV head of one tile of kRows query rows of one
// sequence (row r = new token r / group, query head r % group of the KV head);
// its units are runs of `unit` granules that some row of the tile sees, after
// `head_units` that stand for what a work costs besides its granules; at least
// one (a tile that sees nothing still writes its rows). The works of a launch
// in order (sequence, tile, head) and their units form one list, from which
// every CTA takes an equal part: the lengths are read on the device, so ragged
// batches, and graphs replayed with other lengths, stay balanced.
// ---------------------------------------------------------------------------
struct Span {
  int32_t g0, n;  // first granule, number of granules
};
template <int kRows>
NVFP4_DEVINL Span tile_span(const AttnArgs& a, const KvSeq& s, int tile) {
  const int32_t rows = s.rows * a.group;
  const int32_t r1 = rows - tile * kRows < kRows ? rows : (tile + 1) * kRows;
  const int32_t first = a.by_group.divide(tile * kRows), last = a.by_group.divide(r1 - 1), pos = s.len - s.rows;
  const Visible v0 = visible((int64_t)pos + first, s.len, a.causal, a.window);
  const Visible v1 = visible((int64_t)pos + last, s.len, a.causal, a.window);
  if (v1.hi <= v0.lo) return Span{0, 0};
  const int32_t g0 = v0.lo / kGranule;
  return Span{g0, (v1.hi + kGranule - 1) / kGranule - g0};
}
template <int kRows>
NVFP4_DEVINL int tiles_of(const AttnArgs& a, const KvSeq& s) {
  return (s.rows * a.group + (kRows - 1)) / kRows;
}
NVFP4_DEVINL int units_of(const Span& s, int unit, int head_units) {
  return head_units + (s.n > unit ? (s.n + unit - 1) / unit : 1);
}

constexpr int kStoredSums = 256, kLongList = 64, kLongTiles = 16;

// A CTA's place in the list, moved from work to work.
template <int kRows>
struct WorkCursor {
  KvSeq seq;
  Span span;
  int b, tile, head, n;  // n: units of the work
  int64_t w0;            // the work's first unit
  int unit, head_units;
  NVFP4_DEVINL bool next(const AttnArgs& a) {  // false behind the last work
    w0 += n;
    if (++head < a.ix.hkv) return true;
    head = 0;
    if (++tile >= tiles_of<kRows>(a, seq)) {
      tile = 0;
      do {
        if (++b >= a.ix.batch) return false;
        seq = kv_sequence(a.ix, b, nullptr);
      } while (seq.rows == 0);
    }
    span = tile_span<kRows>(a, seq, tile);
    n = units_of(span, unit, head_units);
    return true;
  }
  // Granules of the work's units [first, last).
  NVFP4_DEVINL void granules(int first, int last, int& g0, int& g1) const {
    g0 = (first < head_units ? 0 : first - head_units) * unit;
    g1 = (last < head_units ? 0 : last - head_units) * unit;
    if (g0 > span.n) g0 = span.n;
    if (g1 > span.n) g1 = span.n;
  }
};

// Where a CTA begins: filled by find_part (its scratch may lie over buffers that
// are not in use yet).
template <int kRows>
struct Part {
  WorkCursor<kRows> cursor;
  int64_t u0, u1, per;  // this CTA's units [u0, u1); units of a CTA
};
struct PartScratch {
  int64_t sums[4][kStoredSums];
  int64_t warp_total[4][32];
  int32_t warp_longest[32];
  int32_t long_seq[kLongList];
  int32_t long_count;
};

// This CTA's part of the list, called by all kThreads threads. What a piece of a
// work costs besides its granules (its queries, its pipeline's start, the warps'
// meeting) is worth kHead units of kFine granules, joining the pieces of a cut
// work Cost::join(pieces) (both measured), and where few CTAs work a granule
// costs Cost::kSparse; so units are chosen among
//   kFine granules and kHead in front of a work: all CTAs take equally much;
//   runs of kLong / 4 or kLong granules: short works are not cut;
//   the run that suits best among those of which every CTA gets one, if there are
//   few works: no CTA has the end of one work and the start of another.
// A thread counts a sequence, a warp one of many tiles.
template <int kRows, int kFine, int kLong, int kHead, int kThreads, class Cost>
NVFP4_DEVINL void find_part(const AttnArgs& a, PartScratch& sh, Part<kRows>& part) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kMid = kLong / 4, kKinds = 3;
  constexpr int kUnit[3] = {kFine, kMid, kLong};
  constexpr int kHeads[3] = {kHead, 0, 0};
  constexpr float kPieceCost = kHead;  // in units of kFine
  constexpr int kSums = kKinds + 1;  // the units of each kind, and the works
  struct Sums {
    int64_t of[kSums];
  };
  int32_t longest = 0;  // granules of the longest work that this thread has counted
  auto count = [&](const KvSeq& s, int t0, int step) {
    Sums u{};
    const int tiles = tiles_of<kRows>(a, s);
    for (int t = t0; t < tiles; t += step) {
      const Span span = tile_span<kRows>(a, s, t);
#pragma unroll
      for (int k = 0; k < kKinds; ++k) u.of[k] += (int64_t)units_of(span, kUnit[k], kHeads[k]) * a.ix.hkv;
      u.of[kKinds] += a.ix.hkv;
      longest = max(longest, span.n);
    }
    return u;
  };
  auto warp_sum = [&](Sums& u) {
    bool small = true;  // 32 summands below 2^26
#pragma unroll
    for (int k = 0; k < kSums; ++k) small = small && u.of[k] < (1 << 26);
    if (__all_sync(0xFFFFFFFFu, small)) {
#pragma unroll
      for (int k = 0; k < kSums; ++k) u.of[k] = __reduce_add_sync(0xFFFFFFFFu, (uint32_t)u.of[k]);
      return;
    }
#pragma unroll
    for (int k = 0; k < kSums; ++k)
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) u.of[k] += __shfl_xor_sync(0xFFFFFFFFu, u.of[k], o);
  };
  const bool few = a.ix.batch <= 32;  // warp 0 alone, a lane for each sequence
  Sums own{};
  KvSeq mine{0, 0, 0};
  if (few && warp == 0) {
    if (lane < a.ix.batch) mine = kv_sequence(a.ix, lane, a.status);
    const bool longer = tiles_of<kRows>(a, mine) > kLongTiles;
    if (!longer) own = count(mine, 0, 1);
    for (unsigned left = __ballot_sync(0xFFFFFFFFu, longer); left; left &= left - 1) {
      const int src = __ffs(left) - 1;
      const KvSeq x{0, __shfl_sync(0xFFFFFFFFu, mine.rows, src), __shfl_sync(0xFFFFFFFFu, mine.len, src)};
      Sums u = count(x, lane, 32);
      warp_sum(u);
      if (lane == src) own = u;
    }
  }
  if (!few) {
    if (tid == 0) sh.long_count = 0;
    __syncthreads();
    Sums sum{};
    for (int b = tid; b < a.ix.batch; b += kThreads) {
      const KvSeq s = kv_sequence(a.ix, b, a.status);
      if (tiles_of<kRows>(a, s) > kLongTiles && b < kStoredSums) {
        const int i = atomicAdd(&sh.long_count, 1);
        if (i < kLongList) {
          sh.long_seq[i] = b;
          continue;
        }
      }
      const Sums u = count(s, 0, 1);
#pragma unroll
      for (int k = 0; k < kSums; ++k) {
        if (b < kStoredSums) sh.sums[k][b] = u.of[k];
        sum.of[k] += u.of[k];
      }
    }
    __syncthreads();
    const int longs = sh.long_count < kLongList ? sh.long_count : kLongList;
    for (int i = warp; i < longs; i += kThreads / 32) {
      const int b = sh.long_seq[i];
      Sums u = count(kv_sequence(a.ix, b, nullptr), lane, 32);
      warp_sum(u);
      if (lane == 0)
#pragma unroll
        for (int k = 0; k < kSums; ++k) {
          sh.sums[k][b] = u.of[k];
          sum.of[k] += u.of[k];
        }
    }
    warp_sum(sum);
    longest = uniform(longest);
    if (lane == 0) sh.warp_longest[warp] = longest;
    if (lane == 0)
#pragma unroll
      for (int k = 0; k < kSums; ++k) sh.warp_total[k][warp] = sum.of[k];
    __syncthreads();
  }
  if (warp == 0) {
    Sums all = own;
    if (!few)
#pragma unroll
      for (int k = 0; k < kSums; ++k) all.of[k] = lane < kThreads / 32 ? sh.warp_total[k][lane] : 0;
    warp_sum(all);
    if (!few) longest = lane < kThreads / 32 ? sh.warp_longest[lane] : 0;
    longest = uniform(longest);
    // (a 64-bit division takes as long as all the rest of this)
    auto parts = [&](int64_t total) {
      return total < (int64_t(1) << 30) ? (int64_t)a.by_grid.divide((int32_t)total + (int)gridDim.x - 1)
                                        : (total + gridDim.x - 1) / gridDim.x;
    };
    int kind = 0, unit = kFine, head_units = kHead;
    int64_t total = all.of[0];
    {
      const int64_t works = all.of[kKinds];
      const float granules = fmaxf((float)(all.of[0] - works * kHead), 1.0f);  // in units of kFine
      const float each = __fdividef(granules, (float)works), share = (float)parts(all.of[0]);
      const float most = (float)longest * (1.0f / kFine);
      // (a CTA may have the end of one work and the start of the next: half a piece more)
      float best = share + 1.5f * kPieceCost + Cost::join(__fdividef(each + kPieceCost, share));
      // CTAs up to this many lie on SMs of their own. (Not half of the grid: six SMs of 148 take a second CTA as the
      // launch's 103rd to 108th, before others have one; 128 CTAs took as long a granule as 296.)
      const float sparse = (float)gridDim.x * (1.0f / 3.0f);
#pragma unroll
      for (int k = 1; k < kKinds; ++k) {
        const float run = fminf((float)kUnit[k] / kFine, most), units = (float)all.of[k];
        const float takes = (float)parts(all.of[k]) * (run * (units <= sparse ? Cost::kSparse : 1.0f) + kPieceCost +
                                                       (all.of[k] > works ? Cost::join(__fdividef(units, (float)works)) : 0.0f));
        if (takes < best) {
          best = takes;
          kind = k;
        }
      }
      if (few && 2 * works <= gridDim.x) {
        // lane x: runs that cut a work into x + 1, or as many as there are CTAs for (ceil(n / unit) over the works is at
        // most granules / unit + works)
        const float least = ceilf(__fdividef(granules, (float)((int)gridDim.x - (int)works))) + 1.0f;
        const float run = fmaxf(least, lane < 31 ? ceilf(__fdividef(each, (float)(lane + 1))) : 0.0f);
        const float pieces = ceilf(__fdividef(each, run));
        const float takes = run * (pieces * (float)works <= sparse ? Cost::kSparse : 1.0f) + kPieceCost +
                            (run < most ? Cost::join(fmaxf(pieces, 2.0f)) : 0.0f);
        const uint32_t least_of = __reduce_min_sync(0xFFFFFFFFu, __float_as_uint(takes));  // positive: ordered as integers
        if (__uint_as_float(least_of) < best) {
          const int src = __ffs(__ballot_sync(0xFFFFFFFFu, __float_as_uint(takes) == least_of)) - 1;
          kind = 3;
          unit = (int)__shfl_sync(0xFFFFFFFFu, run, src) * kFine;
        }
      }
      if (kind) {
        if (kind < 3) unit = kind == 1 ? kMid : kLong;
        head_units = 0;
        if (kind < 3) {
          total = kind == 1 ? all.of[1] : all.of[2];
        } else {
          int64_t u = 0;
          for (int t = 0; t < tiles_of<kRows>(a, mine); ++t)
            u += (int64_t)units_of(tile_span<kRows>(a, mine, t), unit, 0) * a.ix.hkv;
          own.of[0] = u;
          Sums again = own;
          warp_sum(again);
          total = again.of[0];
        }
      }
    }
    const int64_t per = parts(total), u0 = per * blockIdx.x;
    int64_t base = 0;
    // the lane whose part of the list, 32 values on from `base`, holds u0
    auto locate = [&](int64_t v) {
      int64_t incl = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += x;
      }
      const unsigned at = __ballot_sync(0xFFFFFFFFu, base + incl > u0);
      const int src = at ? __ffs(at) - 1 : 31;
      base += __shfl_sync(0xFFFFFFFFu, at ? incl - v : incl, src);
      return at ? src : -1;
    };
    auto of_kind = [&](const Sums& u) { return kind == 1 ? u.of[1] : kind == 2 ? u.of[2] : u.of[0]; };
    int b = -1, tile = -1;
    KvSeq s{0, 0, 0};
    if (u0 < total) {
      if (few) {
        b = locate(of_kind(own));
        if (b >= 0) {
          s.row0 = __shfl_sync(0xFFFFFFFFu, mine.row0, b);
          s.rows = __shfl_sync(0xFFFFFFFFu, mine.rows, b);
          s.len = __shfl_sync(0xFFFFFFFFu, mine.len, b);
        }
      } else {
        for (int b0 = 0; b < 0 && b0 < a.ix.batch; b0 += 32) {
          const int x = b0 + lane;
          int64_t v = 0;
          if (x < kStoredSums && x < a.ix.batch)
            v = sh.sums[kind][x];
          else if (x < a.ix.batch)
            v = of_kind(count(kv_sequence(a.ix, x, nullptr), 0, 1));
          const int src = locate(v);
          if (src >= 0) b = b0 + src;
        }
        if (b >= 0) s = kv_sequence(a.ix, b, nullptr);
      }
      const int tiles = tiles_of<kRows>(a, s);
      if (tiles == 1) tile = 0;
      for (int t0 = 0; tile < 0 && t0 < tiles; t0 += 32) {
        const int x = t0 + lane;
        const int src = locate(x < tiles ? (int64_t)units_of(tile_span<kRows>(a, s, x), unit, head_units) * a.ix.hkv : 0);
        if (src >= 0) tile = t0 + src;
      }
    }
    if (lane == 0) {
      WorkCursor<kRows>& c = part.cursor;
      c.unit = unit;
      c.head_units = head_units;
      part.per = per;
      part.u0 = u0;
      // (no tile: the lengths changed under way, from another stream; no work rather than a wrong one)
      part.u1 = tile < 0 ? u0 : u0 + per < total ? u0 + per : total;
      if (tile >= 0) {
        c.b = b;
        c.tile = tile;
        c.seq = s;
        c.span = tile_span<kRows>(a, s, tile);
        c.n = units_of(c.span, unit, head_units);
        c.head = u0 - base < (int64_t(1) << 31) ? (int)(u0 - base) / c.n : (int)((u0 - base) / c.n);
        c.w0 = base + (int64_t)c.head * c.n;
      }
    }
  }
  __syncthreads();
}

}  // namespace nvfp4
