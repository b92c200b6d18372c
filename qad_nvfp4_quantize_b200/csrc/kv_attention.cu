// nvfp4_paged_attention for few query rows per KV head (decode, drafted
// tokens): out = softmax(scale * Q K^T + mask) V over the paged NVFP4 cache.
//
// Mathematics: one pass over the cached tokens (the running maximum and sum of
// Milakov and Gimelshein, "Online normalizer calculation for softmax", 2018) with
// a maximum m, sum l and unnormalised output O per query row: m' = max(m, s), O =
// O * 2^(m - m') + 2^(s - m') v (scores in units of log2). m is held 7 below the score that set
// it, and O and l are rescaled only when a score exceeds m by more than 15: a
// row's largest p = 2^(s - m) lies between 2^7 and 2^15, FP16's upper end, and
// the sums in FP32 lose nothing.
//
// Bound: HBM, 18*D bytes per 16 tokens and KV head. The rows of one KV head
// (all its query heads, all new tokens of the tile) share each fetched granule.
// Measured, D = 128, 8 rows (single calls on a cold cache): 64 sequences of up to
// 16,384 tokens (739 MB) in 155 to 158 us, 4.7 to 4.8 TB/s; 2 of 131,072 (75 MB)
// in 33 to 35 us (30 back to back). The same loop without its arithmetic, which
// only copies, takes 137 us, without dequantization 145; issue slots are 63 %
// busy, the ALU 54 %. Single tokens over 1,024 cached ones take 14
// us, 4 of them for lengths, page table and queries, one read behind the other,
// and 1 us for each 32 tokens of a warp.
//
// Layout. S^T = K Q^T and O^T = V^T P^T with mma m16n8k16 (FP16 in, FP32 out):
// tokens resp. head dimensions fill the 16 rows, so 8 query rows waste nothing
// and the codes are dequantized straight into the A fragments, each exactly
// once. (A 128-row tcgen05 tile needs 1024 tensor cycles per 128 tokens and
// head; their bytes arrive in 805.) P^T moves from accumulator to B fragment
// by two 8x8 transposes. The order of head dimensions and of tokens within an
// MMA is free as long as both operands agree; it is chosen so that a lane's
// codes are contiguous.
//
// Every warp works alone: pair i of granules of a CTA's span goes to warp i mod
// 8, which has the next pair's bulk copies (18*D bytes each) in flight on its own
// barrier while it works on this one (two pairs ahead changed nothing), and its
// own m, l, O; the warps meet at the end of the span. A work that the cut of the
// work list (kv_attention.cuh) divides leaves partial (m, l, O) in the
// workspace; the last CTA that arrives at the work's counter joins the parts in
// index order (no CTA waits, and the result does not depend on which one is
// last). More than kJoin parts are joined in runs of kJoin first, by the last CTA
// of each run: 74 parts of 4 KB took one CTA 9.7 us, the two rounds take 6.
#include <cuda_fp16.h>

#include "kv_attention.cuh"

namespace nvfp4 {

constexpr int kAttnWarps = 8;
constexpr int kAttnThreads = kAttnWarps * 32;
constexpr int kLongUnit = 384;  // granules: the longest run that is not cut (find_part)
constexpr int kMaxAttnCtas = 320;
constexpr int kJoin = 16;  // parts joined at a time

// Two CTAs for each SM where 128 registers a thread hold the output and the
// queries: 16 rows of 128 dimensions need 230 (with 128 and spills, 16 rows over
// 2,048 cached tokens took 33 us instead of 25).
template <int D, int NT>
constexpr int kCtasPerSm = NT == 1 || D == 64 ? 2 : 1;

// Costs of the work list in the time of a granule: 0.12 us where two CTAs share an
// SM (0.065 where one has it), 0.08 us for 16 rows of 128 dimensions. A piece of a
// work takes about 5 us besides, joining p pieces 1.5 us and 0.25 for each, or 9 us
// in two rounds. Measured, one sequence, 8 KV heads, 8 rows: 2,048 tokens uncut
// 18.5 us, in 4 pieces a head 14.4, in 16 16.4, in 26 18.4; 32,768 in 8 pieces 30.9,
// in 37 26.6.
template <int kPerSm>
struct AttnCost {
  static constexpr int kHead = kPerSm == 2 ? 40 : 60;
  static constexpr float kSparse = kPerSm == 2 ? 0.54f : 1.0f;
  static NVFP4_DEVINL float join(float pieces) {
    const float granules = pieces <= kJoin ? 12.0f + 2.0f * pieces : 75.0f;
    return kPerSm == 2 ? granules : 1.5f * granules;
  }
};

template <int D, int NT>
struct AttnShared {
  static constexpr int kStages = 2;  // pairs of granules that a warp works on or has in flight
  static constexpr int kRows = 8 * NT;
  static constexpr int kPad = D + 8;  // row pitch of the joining buffer
  union {
    uint8_t ring[kAttnWarps][kStages][2 * granule_bytes(D)];
    float join[kAttnWarps][kRows][kPad];
    PartScratch scratch;
  };
  Part<8 * NT> part;
  uint64_t bar[kAttnWarps][kStages];
  float wm[kAttnWarps][kRows], wl[kAttnWarps][kRows];
  float m[kRows], l[kRows];
  float factor[kAttnWarps][kRows];  // of warps with a row of huge scores
  int last;
  volatile int abort;
};

NVFP4_DEVINL void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                            uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
NVFP4_DEVINL uint32_t transpose_8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
NVFP4_DEVINL uint32_t half2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Token (within its granule) of MMA row or depth index i: a lane's four tokens
// of V^T (depths 2t, 2t+1, 2t+8, 2t+9) and the rows of K that eight lanes fetch
// together then fall into different shared-memory banks.
__host__ __device__ constexpr int token_of(int i) {
  return (i & 8) + ((i & 1) ? (((i & 7) >> 1) + 4) ^ 1 : (i & 7) >> 1);
}

template <int D, int NT>
__global__ void __launch_bounds__(kAttnThreads, kCtasPerSm<D, NT>) kv_attention_kernel(const AttnArgs a) {
  using Sh = AttnShared<D, NT>;
  extern __shared__ __align__(128) uint8_t attn_smem[];
  Sh& sh = *reinterpret_cast<Sh*>(attn_smem);
  constexpr int kRows = Sh::kRows, kStages = Sh::kStages, kGB = granule_bytes(D);
  constexpr int kSteps = D / 16;        // k-steps of S, m-tiles of O
  constexpr int kWords = D / 32;        // code words per lane and K row
  const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5), g = lane >> 2, t = lane & 3;

  if (lane == 0)
    for (int i = 0; i < kStages; ++i) mbar_init(&sh.bar[warp][i], 1);
  if (tid == 0) sh.abort = 0;
  fence_barrier_init();

  prefetch_inputs(a, D);
  using Cost = AttnCost<kCtasPerSm<D, NT>>;
  find_part<kRows, 1, kLongUnit, Cost::kHead, kAttnThreads, Cost>(a, sh.scratch, sh.part);
  const int64_t u0 = sh.part.u0, u1 = sh.part.u1, per = sh.part.per;
  if (u0 >= u1) return;
  WorkCursor<kRows> w = sh.part.cursor;
  fence_proxy_async_smem();
  __syncthreads();  // the search's scratch lies over the ring
  uint32_t phase = 0;  // parity bit of each stage of this warp's ring
  auto wait = [&](uint64_t* bar, uint32_t parity) { return wait_bounded(bar, parity, &sh.abort, a.wait_cycles); };
  const float kg = *a.k_g, vg = *a.v_g;

  for (int64_t u = u0;;) {
    const int unit0 = (int)(u - w.w0), unit1 = (int)(u1 - w.w0 < w.n ? u1 - w.w0 : w.n);
    const bool whole_work = unit0 == 0 && unit1 == w.n;
    u = w.w0 + unit1;
    const KvSeq& seq = w.seq;
    const int tile = w.tile, head = w.head, b = w.b;
    int j0, j1;  // granules
    w.granules(unit0, unit1, j0, j1);

    // ---- the queries' rows are on their way first: row r = tile*kRows + 8*nt + g of the head's rows
    const int32_t nrows = seq.rows * a.group;
    uint32_t raw[NT][D / 8];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int32_t r = tile * kRows + 8 * nt + g;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) raw[nt][i] = 0;
      if (r < nrows) {
        const int32_t tok = a.by_group.divide(r), hq = head * a.group + r - tok * a.group;
        const uint4* q4 =
            reinterpret_cast<const uint4*>(a.q + (seq.row0 + tok) * a.q_stride + (int64_t)hq * D + t * (D / 4));
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const uint4 v = ld_stream(q4 + i);
          raw[nt][4 * i] = v.x; raw[nt][4 * i + 1] = v.y; raw[nt][4 * i + 2] = v.z; raw[nt][4 * i + 3] = v.w;
        }
      }
    }

    // ---- this warp's pairs of granules j0 + 2*(warp + 8*i) and the next one; the first ones are fetched while the
    // queries are prepared
    const int cnt = uniform(w.span.n > 0 && j1 - j0 > 2 * warp ? (j1 - j0 - 2 * warp + 2 * kAttnWarps - 1) / (2 * kAttnWarps) : 0);
    const int gfirst = w.span.g0 + j0 + 2 * warp, gend = w.span.g0 + j1;
    const int32_t* table = a.ix.table + (int64_t)b * a.ix.width;
    const int64_t page_bytes = ((int64_t)a.ix.hkv << a.ix.gshift) * kGB;
    const uint8_t* of_head = a.pages + ((int64_t)head << a.ix.gshift) * kGB;
    // Lane x of a block of 16 pairs looks after granule x & 1 of pair x >> 1: where it lies, and whether it is there
    // (within the span, on a page of the pool; else its tokens count as masked).
    const uint8_t* from = nullptr;
    uint32_t there = 0, there_next = 0;
    auto look_up = [&](int i0) {
      const int i = i0 + (lane >> 1), gi = gfirst + 2 * kAttnWarps * i + (lane & 1);
      bool good = i < cnt && gi < gend && NVFP4_IN_BOUNDS(gi >> a.ix.gshift, a.ix.width, a.status);
      if (good) {
        const int32_t p = table[gi >> a.ix.gshift];
        good = p >= 0 && p < a.ix.num_pages;
        if (!good) record_status(a.status, NVFP4_ERR_PAGE);
        int64_t at = p * page_bytes + (int64_t)(gi & ((1 << a.ix.gshift) - 1)) * kGB;
        if (!NVFP4_IN_BOUNDS(at + kGB - 1, good ? a.ix.num_pages * page_bytes : at + kGB, a.status)) at = 0;
        from = of_head + at;
      }
      there_next = __ballot_sync(0xFFFFFFFFu, good);
    };
    auto issue = [&](int i, int st, bool withheld) {  // called by the whole warp, i in order
      if ((i & 15) == 0) look_up(i);
      const uint32_t two = (there_next >> (2 * (i & 15))) & 3u;
      if (two == 0) return;
      if (lane == 0) mbar_arrive_expect_tx(&sh.bar[warp][st], (uint32_t)__popc(two) * kGB);
      __syncwarp();
      if (!withheld && (lane >> 1) == (i & 15) && ((there_next >> lane) & 1u))
        bulk_load(sh.ring[warp][st] + (lane & 1) * kGB, from, kGB, &sh.bar[warp][st]);
    };
    int ahead = 0, st_ahead = 0, st = 0;
    for (; ahead < cnt && ahead < kStages - 1; ++ahead) {
      issue(ahead, st_ahead++, ahead < a.withheld);
      if ((ahead & 15) == 0) there = there_next;
    }

    // ---- queries: B fragments of Q^T
    uint32_t qf[NT][2 * kSteps];
    float factor[NT][2];        // score units of columns 2t, 2t+1
    int32_t lo[NT][2], hi[NT][2];
    int32_t all_lo = 0, all_hi = 0x7FFFFFFF;  // tokens that every row of the tile sees
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      uint32_t mx = 0;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) mx = max(mx, mag_max_halves(raw[nt][i]));
      mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
      mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
      const int ex = query_exponent(__uint_as_float(mx << 16));
#pragma unroll
      for (int e = 0; e < 4 * kWords; ++e)
        qf[nt][e] = half2_bits(scale_exp2(__uint_as_float(raw[nt][e] << 16), ex),
                               scale_exp2(__uint_as_float(raw[nt][e] & 0xFFFF0000u), ex));
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int32_t rc = tile * kRows + 8 * nt + 2 * t + c;
        const int ec = __shfl_sync(0xFFFFFFFFu, ex, (2 * t + c) * 4);
        // not zero: a masked score is -Inf before it is multiplied
        factor[nt][c] = fmaxf(scale_exp2(a.scale * kg * kLog2e, kValueExp - ec), 1.17549435e-38f);
        Visible v{0, 0};
        if (rc < nrows) v = visible(seq.len - seq.rows + a.by_group.divide(rc), seq.len, a.causal, a.window);
        lo[nt][c] = v.lo;
        hi[nt][c] = v.hi;
        if (rc < nrows) {
          all_lo = max(all_lo, v.lo);
          all_hi = min(all_hi, v.hi);
        }
      }
    }
    bool huge = false;  // some row's scores are multiplied by its factor before the maximum, not with it
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) huge |= factor[nt][0] > kHugeFactor<D> || factor[nt][1] > kHugeFactor<D>;
    huge = __any_sync(0xFFFFFFFFu, huge);
    if (huge) {
      __syncwarp();
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const bool of_row = factor[nt][c] > kHugeFactor<D>;
          sh.factor[warp][8 * nt + 2 * t + c] = of_row ? factor[nt][c] : 1.0f;
          if (of_row) factor[nt][c] = 1.0f;
        }
      __syncwarp();
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      all_lo = max(all_lo, __shfl_xor_sync(0xFFFFFFFFu, all_lo, o));
      all_hi = min(all_hi, __shfl_xor_sync(0xFFFFFFFFu, all_hi, o));
    }

    float m[NT][2], l[NT][2], o[NT][kSteps][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = kStartMax;
      l[nt][0] = l[nt][1] = 0.0f;
#pragma unroll
      for (int i = 0; i < kSteps; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.0f;
    }

    bool ok = true;
    for (int i = 0; i < cnt; ++i) {
      if ((i & 15) == 0) there = there_next;  // the look-up of this block ran at most kStages - 1 pairs ago
      const uint32_t two = (there >> (2 * (i & 15))) & 3u;
      if (ahead < cnt) {  // into the stage that the last trip has read
        issue(ahead++, st_ahead, false);
        if (++st_ahead == kStages) st_ahead = 0;
      }
      if (two) {
        if (!(ok = wait(&sh.bar[warp][st], (phase >> st) & 1u))) break;
        phase ^= 1u << st;
      }
      const uint8_t* gr = sh.ring[warp][st];
      if (++st == kStages) st = 0;
      if (two == 0) continue;

      // S^T of 32 tokens
      float s[NT][2][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[nt][y][e] = 0.0f;
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        uint32_t wa[kWords], wb[kWords];  // rows g and g + 8
        const uint8_t* k0 = gr + y * kGB;
        const uint8_t* ka = k0 + token_of(g) * (D / 2) + t * (D / 8);
        const uint8_t* kb = k0 + token_of(g + 8) * (D / 2) + t * (D / 8);
        uint32_t sa, sb;  // scale bytes of the lane's D/4 dimensions (two blocks, or one)
        if constexpr (D == 128) {
          const uint4 u = *reinterpret_cast<const uint4*>(ka), v = *reinterpret_cast<const uint4*>(kb);
          wa[0] = u.x; wa[1] = u.y; wa[2] = u.z; wa[3] = u.w;
          wb[0] = v.x; wb[1] = v.y; wb[2] = v.z; wb[3] = v.w;
          sa = *reinterpret_cast<const uint16_t*>(k0 + 8 * D + token_of(g) * 8 + 2 * t);
          sb = *reinterpret_cast<const uint16_t*>(k0 + 8 * D + token_of(g + 8) * 8 + 2 * t);
        } else {
          const uint2 u = *reinterpret_cast<const uint2*>(ka), v = *reinterpret_cast<const uint2*>(kb);
          wa[0] = u.x; wa[1] = u.y;
          wb[0] = v.x; wb[1] = v.y;
          sa = k0[8 * D + token_of(g) * 4 + t];
          sb = k0[8 * D + token_of(g + 8) * 4 + t];
        }
#pragma unroll
        for (int blk = 0; blk < D / 64; ++blk) {
          const uint32_t fa = scales_to_half(__byte_perm(sa, 0, blk ? 0x4141 : 0x4040));
          const uint32_t fb = scales_to_half(__byte_perm(sb, 0, blk ? 0x4141 : 0x4040));
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int x = 2 * blk + h;
            uint32_t pa[4], pb[4];
            codes_to_half(wa[x], pa);
            codes_to_half(wb[x], pb);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              pa[e] = hmul2(pa[e], fa);
              pb[e] = hmul2(pb[e], fb);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma_16816(s[nt][y], pa[0], pb[0], pa[1], pb[1], qf[nt][4 * x], qf[nt][4 * x + 1]);
              mma_16816(s[nt][y], pa[2], pb[2], pa[3], pb[3], qf[nt][4 * x + 2], qf[nt][4 * x + 3]);
            }
          }
        }
      }

      // mask, running maximum (m in log2 units; scores become that with the row's factor in the exponent's FMA)
      const int tok0 = (gfirst + 2 * kAttnWarps * i) * kGranule;
      const bool whole = tok0 >= all_lo && tok0 + 2 * kGranule <= all_hi && two == 3u;
      bool grow = false;
      if (!whole) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int tk = tok0 + kGranule * y + token_of(g + (e & 2) * 4), c = e & 1;
              if (tk < lo[nt][c] || tk >= hi[nt][c] || !((two >> y) & 1u)) s[nt][y][e] = -INFINITY;
            }
      }
      if (huge) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float f = sh.factor[warp][8 * nt + 2 * t + c];
            s[nt][0][c] *= f;
            s[nt][0][c + 2] *= f;
            s[nt][1][c] *= f;
            s[nt][1][c + 2] *= f;
          }
      }
      float top[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          top[nt][c] = fmaxf(max3(s[nt][0][c], s[nt][0][c + 2], s[nt][1][c]), s[nt][1][c + 2]) * factor[nt][c];
          grow |= exceeds(top[nt][c], m[nt][c]);
        }
      if (__any_sync(0xFFFFFFFFu, grow)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float mx = top[nt][c];
            mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 16));
            const float m1 = new_max(mx, m[nt][c]);
            const float f = m[nt][c] == kStartMax ? 0.0f : ex2(m[nt][c] - m1);
            m[nt][c] = m1;
            l[nt][c] *= f;
#pragma unroll
            for (int x = 0; x < kSteps; ++x) {
              o[nt][x][c] *= f;
              o[nt][x][c + 2] *= f;
            }
          }
      }
      // P^T as B fragments: FP16 rounds p to 2^-11 of itself from 2^-14 on, below to 2^-25 (2^-32 of the largest p)
      uint32_t pf[NT][2][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          float p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) p[e] = ex2(__fmaf_rn(s[nt][y][e], factor[nt][e & 1], -m[nt][e & 1]));
          l[nt][0] += p[0] + p[2];
          l[nt][1] += p[1] + p[3];
          pf[nt][y][0] = transpose_8x8(half2_bits(p[0], p[1]));
          pf[nt][y][1] = transpose_8x8(half2_bits(p[2], p[3]));
        }
      }

      // O^T += V^T P^T
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const uint8_t* v0 = gr + y * kGB + 9 * D;
        const uint8_t* vs = gr + y * kGB + 17 * D;
        constexpr int kVWords = D / 64;
        uint32_t v[4][kVWords], f[2];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int tk = token_of(2 * t + (k & 1) + (k & 2) * 4);
          if constexpr (D == 128) {
            const uint2 u = *reinterpret_cast<const uint2*>(v0 + tk * 64 + 8 * g);
            v[k][0] = u.x;
            v[k][1] = u.y;
          } else {
            v[k][0] = *reinterpret_cast<const uint32_t*>(v0 + tk * 32 + 4 * g);
          }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int ta = token_of(2 * t + 8 * k), tb = token_of(2 * t + 1 + 8 * k);
          const uint32_t u = D == 128 ? vs[ta * 8 + g] : vs[ta * 4 + (g >> 1)];
          const uint32_t z = D == 128 ? vs[tb * 8 + g] : vs[tb * 4 + (g >> 1)];
          f[k] = scales_to_half(u | (z << 16));
        }
#pragma unroll
        for (int x = 0; x < kVWords; ++x) {  // eight dimensions of the lane's run at a time
          // the tokens' nibbles side by side: even dimensions, then odd ones, of two tokens in each byte
          uint32_t pa[2][4], pb[2][4];
          codes_to_half((v[0][x] & 0x0F0F0F0Fu) | ((v[1][x] << 4) & 0xF0F0F0F0u), pa[0]);
          codes_to_half(((v[0][x] >> 4) & 0x0F0F0F0Fu) | (v[1][x] & 0xF0F0F0F0u), pa[1]);
          codes_to_half((v[2][x] & 0x0F0F0F0Fu) | ((v[3][x] << 4) & 0xF0F0F0F0u), pb[0]);
          codes_to_half(((v[2][x] >> 4) & 0x0F0F0F0Fu) | (v[3][x] & 0xF0F0F0F0u), pb[1]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {  // m-tile: dimensions 8x + 2e (rows 0..7) and 8x + 2e + 1 (rows 8..15)
            const uint32_t a0 = hmul2(pa[0][e], f[0]), a1 = hmul2(pa[1][e], f[0]);
            const uint32_t a2 = hmul2(pb[0][e], f[1]), a3 = hmul2(pb[1][e], f[1]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_16816(o[nt][4 * x + e], a0, a1, a2, a3, pf[nt][y][0], pf[nt][y][1]);
          }
        }
      }
      __syncwarp();  // the stage may be refilled
    }

    if (!ok) {
      if (lane == 0) record_status(a.status, NVFP4_ERR_TIMEOUT);
      for (int x = 0; x < kStages; ++x) settle(&sh.bar[warp][x], (phase >> x) & 1u);
    }

    // ---- the warps' parts meet. (A row with a score of NaN or +Inf, from a query that holds NaN or Inf, shows it in its
    // sum l alone: l is multiplied by 0, never left out, where a part saw nothing.)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c)
        if (m[nt][c] == kStartMax) m[nt][c] = -INFINITY;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float x = l[nt][c];
        x += __shfl_xor_sync(0xFFFFFFFFu, x, 4);
        x += __shfl_xor_sync(0xFFFFFFFFu, x, 8);
        x += __shfl_xor_sync(0xFFFFFFFFu, x, 16);
        if (g == 0) {
          sh.wm[warp][8 * nt + 2 * t + c] = m[nt][c];
          sh.wl[warp][8 * nt + 2 * t + c] = x;
        }
      }
    __syncthreads();  // every warp has read its ring: the joining buffer may take its place
    if (sh.abort) return;  // (set before this barrier only: the next wait lies behind others)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int row = 8 * nt + 2 * t + c;
        float mt = -INFINITY;
#pragma unroll
        for (int w = 0; w < kAttnWarps; ++w) mt = fmaxf(mt, sh.wm[w][row]);
        const float f = m[nt][c] == -INFINITY ? 0.0f : ex2(m[nt][c] - mt);
#pragma unroll
        for (int j = 0; j < kSteps; ++j)  // dimensions 2j, 2j+1 of the run of D/8 that starts at g*D/8
          *reinterpret_cast<float2*>(&sh.join[warp][row][g * (D / 8) + 2 * j]) =
              make_float2(o[nt][j][c] * f, o[nt][j][c + 2] * f);
      }
    if (tid < kRows) {
      float mt = -INFINITY, lt = 0.0f;
      for (int w = 0; w < kAttnWarps; ++w) mt = fmaxf(mt, sh.wm[w][tid]);
      for (int w = 0; w < kAttnWarps; ++w)
        lt += sh.wl[w][tid] * (sh.wm[w][tid] == -INFINITY ? 0.0f : ex2(sh.wm[w][tid] - mt));
      sh.m[tid] = mt;
      sh.l[tid] = lt;
    }
    __syncthreads();

    // ---- a whole work is written out; a part goes to the workspace, and the last part joins them
    struct Sums {
      float4 o;  // unnormalised, of 4 dimensions of a row
      float m, l;
    };
    auto for_each = [&](auto&& f) {  // f(row, d): this thread's runs of 4 dimensions
#pragma unroll
      for (int e0 = 0; e0 < kRows * (D / 4); e0 += kAttnThreads) {
        const int e = e0 + tid;
        if (kRows * (D / 4) >= kAttnThreads || e < kRows * (D / 4)) f(e / (D / 4), (e % (D / 4)) * 4);
      }
    };
    auto write_out = [&](int row, int d, const Sums& x) {
      const int32_t r = tile * kRows + row;
      if (r >= nrows) return;
      const int32_t tok = a.by_group.divide(r), hq = head * a.group + r - tok * a.group;
      const int64_t at = (seq.row0 + tok) * a.ix.hkv * a.group + hq;
      const float f = x.l == 0.0f ? 0.0f : output_factor(vg, x.l);  // no visible token: zeros
      if (!NVFP4_IN_BOUNDS(at, a.ix.total * a.ix.hkv * a.group, a.status)) return;
      *reinterpret_cast<uint2*>(a.out + at * D + d) =
          make_uint2(f32x2_to_bf16x2(x.o.x * f, x.o.y * f), f32x2_to_bf16x2(x.o.z * f, x.o.w * f));
      if (a.lse && d == 0) a.lse[at] = x.l == 0.0f ? -INFINITY : (x.m + log2f(x.l)) * kLn2;
    };
    constexpr int kPart = kRows * (D + 2);  // O, then m and l of each row
    auto write_part = [&](float* part, int row, int d, const Sums& x) {
      *reinterpret_cast<float4*>(part + row * D + d) = x.o;
      if (d == 0) {
        part[kRows * D + row] = x.m;
        part[kRows * D + kRows + row] = x.l;
      }
    };
    auto of_warps = [&](int row, int d) {
      Sums x{make_float4(0.0f, 0.0f, 0.0f, 0.0f), sh.m[row], sh.l[row]};
#pragma unroll
      for (int w2 = 0; w2 < kAttnWarps; ++w2) {
        const float4 y = *reinterpret_cast<const float4*>(&sh.join[w2][row][d]);
        x.o.x += y.x;
        x.o.y += y.y;
        x.o.z += y.z;
        x.o.w += y.w;
      }
      return x;
    };
    if (whole_work) {
      for_each([&](int row, int d) { write_out(row, d, of_warps(row, d)); });
    } else {
      // A CTA has two places: the second for the part that begins a work, the first for a later part of one.
      auto place = [&](int cta, int which) { return a.partial + (2 * (int64_t)cta + which) * kPart; };
      float* part = place(blockIdx.x, unit0 == 0 ? 1 : 0);
      for_each([&](int row, int d) { write_part(part, row, d, of_warps(row, d)); });
      __syncthreads();
      const int c0 = (int)(w.w0 / per), np = (int)((w.w0 + w.n - 1) / per) - c0 + 1;  // the CTAs that share the work
      // What a run of parts from `first` on is joined to: the second place of a CTA that has this work only.
      auto joined = [&](int first) { return place(c0 + (first > 0 ? first : 1), 1); };
      for (int round = np > kJoin ? 0 : 1; round < 2; ++round) {
        const bool runs = round == 1 && np > kJoin;
        const int first = round == 0 ? ((int)blockIdx.x - c0) / kJoin * kJoin : 0;
        const int n = round == 0 ? min(kJoin, np - first) : runs ? (np + kJoin - 1) / kJoin : np;
        if (n == 1) continue;  // a run of one part is joined already
        if (tid == 0) sh.last = arrive_last(a.counters + (round == 0 ? kMaxAttnCtas : 0) + c0 + first, n - 1);
        __syncthreads();
        if (!sh.last) break;
        auto nth = [&](int i) -> const float* {
          const int c = runs ? i * kJoin : first + i;
          return runs && c + 1 < np ? joined(c) : place(c0 + c, c == 0 ? 1 : 0);
        };
        // All of kBatch parts in flight, joined with a running maximum in the parts' order. (Maxima first and sums behind a
        // barrier: 64 sequences of up to 16,384 tokens took 158 us, not 154.)
        for_each([&](int row, int d) {
          constexpr int kBatch = 8;
          Sums x{make_float4(0.0f, 0.0f, 0.0f, 0.0f), -INFINITY, 0.0f};
          for (int i = 0; i < n; i += kBatch) {
            Sums y[kBatch];
#pragma unroll
            for (int c = 0; c < kBatch; ++c) {
              y[c] = Sums{make_float4(0.0f, 0.0f, 0.0f, 0.0f), -INFINITY, 0.0f};
              if (i + c < n) {
                const float* from = nth(i + c);
                y[c].o = __ldcg(reinterpret_cast<const float4*>(from + row * D + d));
                y[c].m = __ldcg(from + kRows * D + row);
                y[c].l = __ldcg(from + kRows * D + kRows + row);
              }
            }
            float mt = fmaxf(x.m, kStartMax);  // finite also where no token has been seen so far
#pragma unroll
            for (int c = 0; c < kBatch; ++c) mt = fmaxf(mt, y[c].m);
            auto add = [&](Sums& to, const Sums& z) {
              const float f = ex2(z.m - mt);  // 0 for a part without a visible token: its sums are zeros, or l is NaN
              to.o.x += z.o.x * f;
              to.o.y += z.o.y * f;
              to.o.z += z.o.z * f;
              to.o.w += z.o.w * f;
              to.l += z.l * f;
            };
            Sums z{make_float4(0.0f, 0.0f, 0.0f, 0.0f), mt, 0.0f};
            add(z, x);
#pragma unroll
            for (int c = 0; c < kBatch; ++c) add(z, y[c]);
            x = z;
          }
          if (round == 1)
            write_out(row, d, x);
          else
            write_part(joined(first), row, d, x);
        });
        __syncthreads();
      }
    }
    fence_proxy_async_smem();  // the joining buffer's place is filled by bulk copies again
    __syncthreads();
    if (u >= u1 || !w.next(a)) break;
  }
}

// Counters of works, from kMaxAttnCtas on those of runs of kJoin parts; the 4,096 bytes that callers zero-fill.
constexpr int kCounters = 1024;
static_assert(2 * kMaxAttnCtas <= kCounters, "counters");
constexpr int kPartFloats = 16 * (128 + 2);

size_t kv_attention_workspace_bytes() {
  const size_t rows = (size_t)2 * kMaxAttnCtas * kPartFloats, tiles = kv_prefill_partial_floats();
  return kCounters * sizeof(int32_t) + (rows > tiles ? rows : tiles) * sizeof(float);
}

template <int D, int NT>
cudaError_t launch_rows(AttnArgs a, int num_sms, cudaStream_t s) {
  using Sh = AttnShared<D, NT>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void*>(&kv_attention_kernel<D, NT>), sizeof(Sh), done);
  if (e != cudaSuccess) return e;
  const int64_t want = kCtasPerSm<D, NT> * (int64_t)num_sms;
  const int grid = (int)(want < kMaxAttnCtas ? want : kMaxAttnCtas);
  a.by_grid = Divisor(grid);
  note_launch();
  kv_attention_kernel<D, NT><<<grid, kAttnThreads, sizeof(Sh), s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_kv_attention(AttnArgs a, int D, int64_t max_q, void* workspace, int num_sms, cudaStream_t s) {
  if (a.ix.total == 0 || a.ix.batch == 0) return cudaSuccess;
  a.by_group = Divisor(a.group);
  a.counters = static_cast<int32_t*>(workspace);
  a.partial = reinterpret_cast<float*>(a.counters + kCounters);
  // Rows of a KV head: up to 8 a tile of 8, up to 32 tiles of 16, above tiles of 256 on tcgen05. Measured with 32
  // sequences of 8,192 tokens, 4 KV heads of 128: 8 rows 48 us in a tile of 8 and 64 in one of 16; 16 rows 84, 64 and
  // 122 us on tcgen05; 32 rows 139, 105 and 123; with 64 sequences of 512 tokens and 64 rows 131, 133 and 57.
  if (max_q == 0 || max_q > 32 || max_q * a.group > 32) return launch_kv_prefill(a, D, num_sms, s);
  const bool one = max_q * a.group <= 8;
  if (D == 128) return one ? launch_rows<128, 1>(a, num_sms, s) : launch_rows<128, 2>(a, num_sms, s);
  return one ? launch_rows<64, 1>(a, num_sms, s) : launch_rows<64, 2>(a, num_sms, s);
}

}  // namespace nvfp4
