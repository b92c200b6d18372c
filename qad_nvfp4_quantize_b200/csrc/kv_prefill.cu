// nvfp4_paged_attention for many query rows per KV head (prompts, chunks):
// the same mathematics as kv_attention.cu on tcgen05 tensor cores.
//
// Bound: the tensor pipe (4*D FLOP per row and token), the 2^x unit (16 a cycle
// and SM: as long as the two MMAs of a 128 x 128 tile with D = 128) and the
// issue slots that dequantization and softmax share. Measured, 32 heads of 128:
// 4,096 tokens over 12,288 cached ones, 4 KV heads (687 GFLOP), in 645 to 680 us by
// itself (up to 1.06 PFLOP/s), 705 to 713 back to back under the power limit; 4
// chunks of up to 512 over 16,384, 8 KV heads (315 GFLOP), in 338 to 356 us. Shared
// memory is then 76 % busy (49 % the MMAs' operands, 27 % loads and stores), the
// tensor pipe 50 % and the issue slots 52 %.
//
// One CTA per SM walks its part of the work list; a work is 256 query rows (two
// tiles of 128) of one KV head against its cached tokens, 128 at a time.
//   warps 0..3, 4..7   softmax of row tile 0 and 1, a thread per row, in steps
//                      of 64 tokens: scores from tensor memory, p = 2^(s*c - m)
//                      as FP16 pairs back into the same columns, the output's
//                      rescaling and the epilogue;
//   warp 14            bulk copies of the codes, kStages tiles ahead;
//   warps 8..11        dequantization: K and V as FP16 rows of 64 dimensions,
//                      128-byte swizzled, into a ring of three tiles (K0 V0 K1
//                      V1 ...);
//   warps 12, 13       issue the MMAs of row tile 0 and 1: S = Q K^T (K-major
//                      operands), O += P V (P from tensor memory, V with its
//                      64-dimension runs as the MN-major operand).
// Tensor memory, for each row tile: two S/P buffers of 64 columns and O of D.
// While the softmax works on step t, S of step t + 1 is there already; S of
// step t + 2 is issued when P V of step t is complete (its columns hold P).
// What this buys: with one S of 128 tokens per row tile the softmax waited for
// P V and the next S each time (4,096 over 12,288: 741 us). Two row tiles, not
// one, because each dequantized tile then serves 256 rows.
//
// The running maximum m is held 7 below the score that set it and may lag by 8
// (in log2 units): a row takes a new one, and O is rescaled, only when a score
// exceeds m by more than 15, so that p stays within FP16 and most steps leave O
// alone.
#include <cuda_fp16.h>

#include "kv_attention.cuh"

namespace nvfp4 {

constexpr int kPreThreads = 512;
constexpr int kPreRows = 256;
constexpr int kTileTokens = 128;
constexpr int kUnitGranules = kTileTokens / kGranule;
// Of every six pairs of weights one comes from the FMA pipe instead of the 2^x unit. Measured, 4,096 over 12,288: none
// 673 us, one of eight 660, of six 651, of four 684, of two 751.
constexpr int kPolyEvery = 6;

// Costs of the work list (find_part) in the time of a tile of 128 tokens: joining p pieces 3 + p / 2; a piece besides its
// tiles 2 (kHead of the call); runs of at most 16 tiles are not cut (4 and 64 as the limit gave the same times within 1 %).
// Measured, 32 heads over 8 KV heads of 128, with joins for nothing, as they are here, and at four times that: 16 tokens
// over 4,000 49, 37 and 34 us, over 16,000 62, 56 and 56; 16 sequences of 64 tokens over up to 2,000 71, 71 and 53; 512
// tokens over 4,000 72 each; 4 chunks of up to 512 over 16,384 336, 337 and 337. A piece at 1, 2 and 8: 16 sequences of 64
// 70, 71 and 52; 512 over 4,000 71, 72 and 62; 2,048 over 8,000 248, 249 and 253; 64 over 16,000, four of them, 102, 104
// and 107. No pair is best at all of these.
struct PreCost {
  static constexpr float kSparse = 1.0f;
  static NVFP4_DEVINL float join(float pieces) { return 3.0f + 0.5f * pieces; }
};

template <int D>
struct PreShared {
  static constexpr int kStages = 3;  // tiles of codes in flight
  static constexpr int kTiles = 3;
  static constexpr int kTile = kTileTokens * D * 2;  // bytes of an FP16 tile
  uint8_t kv[kTiles][kTile];                         // K and V tiles in turn: K0 V0 K1 V1 ...
  union {
    uint8_t q[2][kTile];
    PartScratch scratch;
  };
  uint8_t codes[kStages][kUnitGranules][granule_bytes(D)];
  uint64_t codes_full[kStages], codes_empty[kStages];
  uint32_t there[kStages];  // bit g: granule g of the tile is there (within the span, on a page of the pool)
  uint64_t full[kTiles], empty[kTiles];
  uint64_t q_full[2], s_full[2][2], p_full[2][2], pv_done[2][2], group[2], drain[2];
  Part<kPreRows> part;
  WorkCursor<kPreRows> cursor[kPreThreads / 32];  // one per warp: no register is spent on it
  float factor[kPreRows];  // of warps with a row of huge scores
  uint32_t tmem;
  int last[2];
  volatile int abort;
};

// kind::f16 instruction descriptor: D FP32, A and B FP16, M = 128.
__host__ __device__ constexpr uint32_t idesc_f16(int n, bool b_mn_major) {
  return (1u << 4) | (b_mn_major ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}
// A run of MMAs issued by one elected lane of a converged warp: one statement,
// so that the lane is elected once.
// S[tmem] = Q K^T over D dimensions: 32 bytes a step within a 64-dimension
// half, halves 16 KB (1024 descriptor units) apart.
template <int D>
NVFP4_DEVINL void mma_scores(uint32_t d, uint64_t q, uint64_t k, uint32_t idesc) {
  if constexpr (D == 128) {
    asm volatile(
        "{\n\t.reg .pred e, t, z;\n\t.reg .b64 a, b;\n\t.reg .b32 c;\n\t"
        "elect.sync _|e, 0xffffffff;\n\tsetp.eq.u32 t, 0, 0;\n\tsetp.ne.u32 z, 0, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, z;\n\t"
        "add.s64 a, %1, 2;\n\tadd.s64 b, %2, 2;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
        "add.s64 a, %1, 4;\n\tadd.s64 b, %2, 4;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
        "add.s64 a, %1, 6;\n\tadd.s64 b, %2, 6;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
        "add.s64 a, %1, 1024;\n\tadd.s64 b, %2, 1024;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
        "add.s64 a, %1, 1026;\n\tadd.s64 b, %2, 1026;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
        "add.s64 a, %1, 1028;\n\tadd.s64 b, %2, 1028;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
        "add.s64 a, %1, 1030;\n\tadd.s64 b, %2, 1030;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
        "}"
        ::"r"(d), "l"(q), "l"(k), "r"(idesc)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred e, t, z;\n\t.reg .b64 a, b;\n\t.reg .b32 c;\n\t"
        "elect.sync _|e, 0xffffffff;\n\tsetp.eq.u32 t, 0, 0;\n\tsetp.ne.u32 z, 0, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, z;\n\t"
        "add.s64 a, %1, 2;\n\tadd.s64 b, %2, 2;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
        "add.s64 a, %1, 4;\n\tadd.s64 b, %2, 4;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
        "add.s64 a, %1, 6;\n\tadd.s64 b, %2, 6;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
        "}"
        ::"r"(d), "l"(q), "l"(k), "r"(idesc)
        : "memory");
  }
}
// O[tmem] (+)= P V of 64 tokens: P in 8 columns a step, V in two groups of
// eight rows of 128 bytes.
NVFP4_DEVINL void mma_values(uint32_t d, uint32_t p, uint64_t v, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred e, t, z;\n\t.reg .b64 a, b;\n\t.reg .b32 c;\n\t"
      "elect.sync _|e, 0xffffffff;\n\tsetp.eq.u32 t, 0, 0;\n\tsetp.ne.u32 z, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, z;\n\t"
      "add.s32 c, %1, 8;\n\tadd.s64 b, %2, 128;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [c], b, %3, t;\n\t"
      "add.s32 c, %1, 16;\n\tadd.s64 b, %2, 256;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [c], b, %3, t;\n\t"
      "add.s32 c, %1, 24;\n\tadd.s64 b, %2, 384;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [c], b, %3, t;\n\t"
      "}"
      ::"r"(d), "r"(p), "l"(v), "r"(idesc), "r"(acc)
      : "memory");
}
// Columns of this warp's 32 tensor-memory lanes, with the wait: one statement,
// so that the compiler moves or spills no register of a load under way.
NVFP4_DEVINL void tmem_read16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {"
      "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
NVFP4_DEVINL void tmem_read32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
      "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
NVFP4_DEVINL void tmem_read64(uint32_t taddr, uint32_t (&r)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
      "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
      "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
      "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
        "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
        "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
        "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
        "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
      : "r"(taddr)
      : "memory");
}
NVFP4_DEVINL void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {"
      "%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
NVFP4_DEVINL void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
NVFP4_DEVINL f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
NVFP4_DEVINL f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// 2^x of two numbers x < 128 (x <= 15 here) on the FMA pipe: n = x rounded to an integer (by
// adding 1.5 * 2^23), a polynomial for 2^(x - n) on [-1/2, 1/2], n added to the
// exponent (the reduction of Cody and Waite, "Software Manual for the Elementary
// Functions", 1980). Its coefficients are a relative minimax fit of degree 5 (least
// squares, reweighted): off by at most 2^-22 when evaluated in FP32. Arguments
// below -126 give 2^-126, which FP16 rounds to zero.
NVFP4_DEVINL void exp2_poly(f32x2 x, float& r0, float& r1) {
  float x0, x1;
  unpack2(x, x0, x1);
  x = pack2(fmaxf(x0, -126.0f), fmaxf(x1, -126.0f));
  const f32x2 magic = pack2(12582912.0f, 12582912.0f), unmagic = pack2(-12582912.0f, -12582912.0f);
  const f32x2 minus = pack2(-1.0f, -1.0f);
  const f32x2 shifted = add2(x, magic);
  const f32x2 f = fma2(add2(shifted, unmagic), minus, x);
  f32x2 p = pack2(0.001327647f, 0.001327647f);
  p = fma2(p, f, pack2(0.009675541f, 0.009675541f));
  p = fma2(p, f, pack2(0.055507135f, 0.055507135f));
  p = fma2(p, f, pack2(0.2402212f, 0.2402212f));
  p = fma2(p, f, pack2(0.69314694f, 0.69314694f));
  p = fma2(p, f, pack2(1.0000001f, 1.0000001f));
  float p0, p1, n0, n1;
  unpack2(p, p0, p1);
  unpack2(shifted, n0, n1);
  r0 = __uint_as_float(__float_as_uint(p0) + (__float_as_uint(n0) << 23));
  r1 = __uint_as_float(__float_as_uint(p1) + (__float_as_uint(n1) << 23));
}
NVFP4_DEVINL uint32_t half2_of(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Byte of 16-byte chunk c (0..7) of row r of half h (64 dimensions) in a 128-byte-swizzled tile.
NVFP4_DEVINL uint32_t tile_chunk(int h, int r, int c) {
  return (uint32_t)(h * kTileTokens * 128 + r * 128 + ((c ^ (r & 7)) << 4));
}

template <int D>
__global__ void __launch_bounds__(kPreThreads, 1) kv_prefill_kernel(const AttnArgs a) {
  using Sh = PreShared<D>;
  constexpr int kGB = granule_bytes(D), kStages = Sh::kStages;
  extern __shared__ uint8_t pre_smem[];
  Sh& sh = *reinterpret_cast<Sh*>((reinterpret_cast<uintptr_t>(pre_smem) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5);

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sh.codes_full[i], 1);
      mbar_init(&sh.codes_empty[i], 4);
    }
    for (int i = 0; i < Sh::kTiles; ++i) {
      mbar_init(&sh.full[i], 4);
      mbar_init(&sh.empty[i], 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.q_full[i], 4);
      mbar_init(&sh.s_full[i][0], 1);
      mbar_init(&sh.s_full[i][1], 1);
      mbar_init(&sh.p_full[i][0], 4);
      mbar_init(&sh.p_full[i][1], 4);
      mbar_init(&sh.pv_done[i][0], 1);
      mbar_init(&sh.pv_done[i][1], 1);
      mbar_init(&sh.group[i], 4);
      mbar_init(&sh.drain[i], 1);
    }
    sh.abort = 0;
    fence_barrier_init();
  }
  prefetch_inputs(a, D);
  find_part<kPreRows, kUnitGranules, 16 * kUnitGranules, 2, kPreThreads, PreCost>(a, sh.scratch, sh.part);
  if (sh.part.u0 >= sh.part.u1) return;
  const int64_t u0 = sh.part.u0;
  WorkCursor<kPreRows>& w = sh.cursor[warp];
  if (lane == 0) w = sh.part.cursor;
  fence_proxy_async_smem();
  if (warp == 12) {
    tmem_alloc(&sh.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();  // the search's scratch lies over Q
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  auto timed_out = [&]() {
    if (lane == 0) record_status(a.status, NVFP4_ERR_TIMEOUT);
  };
  auto wait = [&](uint64_t* bar, uint32_t parity) { return wait_bounded(bar, parity, &sh.abort, a.wait_cycles); };
  // place of K (2t) or V (2t + 1) in the ring of tiles, and the parity of its turn there
  auto place = [](uint32_t x) { return x % Sh::kTiles; };
  auto turn_of = [](uint32_t x) { return (x / Sh::kTiles) & 1; };
  // units of the work that are this CTA's: its part begins at u0 and at the first unit of every later work
  auto from_unit = [&]() { return (int)(w.w0 < u0 ? u0 - w.w0 : 0); };
  auto to_unit = [&]() { return (int)(sh.part.u1 - w.w0 < w.n ? sh.part.u1 - w.w0 : (int64_t)w.n); };
  // and their tiles of 128 tokens (the reductions make the values warp-uniform to the compiler as well). A part without
  // granules (a work that sees nothing, or a cut in front of the first one) takes the tile behind the work's last,
  // whose tokens are all masked.
  auto tiles_of_part = [&](int& j0, int& j1) {
    int g0, g1;
    w.granules(from_unit(), to_unit(), g0, g1);
    const int behind = (w.span.n + kUnitGranules - 1) / kUnitGranules;
    j0 = uniform(g1 > g0 ? g0 / kUnitGranules : behind);
    j1 = uniform(g1 > g0 ? (g1 + kUnitGranules - 1) / kUnitGranules : behind + 1);
  };
  auto next_work = [&]() {  // the warp's cursor moves on; false at the end of the part
    __syncwarp();
    int more = 0;
    if (lane == 0) more = w.w0 + w.n < sh.part.u1 && w.next(a);
    __syncwarp();
    return __any_sync(0xFFFFFFFFu, more) != 0;
  };

  if (warp < 8) {
    // ------------------------------------------------------------- softmax
    const int i = warp >> 2, wq = warp & 3, row = tid & 127;
    const uint32_t lane_base = (uint32_t)(wq * 32) << 16;
    const uint32_t t_s = tmem + lane_base + i * 128, t_o = tmem + lane_base + 256 + i * D;
    const float kg = *a.k_g, vg = *a.v_g;
    uint32_t steps = 0, meets = 0;
    auto meet = [&]() {  // the four warps of the row tile, with the usual bound
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.group[i]);
      return wait(&sh.group[i], meets++ & 1);
    };
    bool ok = true;
    while (ok) {
      int j0, j1;
      tiles_of_part(j0, j1);
      const int32_t nrows = w.seq.rows * a.group;
      const int32_t r0 = w.tile * kPreRows + i * 128, r = r0 + row;
      if (r0 < nrows) {
        // ---- this thread's query row as FP16, its power of two taken out
        const bool live = r < nrows;
        const int32_t t = a.by_group.divide(r);
        const int64_t tok = w.seq.row0 + t, hq = (int64_t)w.head * a.group + r - t * a.group;
        const uint4* q4 = reinterpret_cast<const uint4*>(a.q + tok * a.q_stride + hq * D);
        uint32_t mx = 0;
        if (live)
#pragma unroll
          for (int c = 0; c < D / 8; ++c) {
            const uint4 x = ld_stream(q4 + c);
            mx = max(max(mx, mag_max_halves(x.x)), max(mag_max_halves(x.y), max(mag_max_halves(x.z), mag_max_halves(x.w))));
          }
        const int ex = query_exponent(__uint_as_float(mx << 16));
#pragma unroll 4
        for (int c = 0; c < D / 8; ++c) {
          uint4 x = make_uint4(0, 0, 0, 0);
          if (live) x = ld_stream(q4 + c);
          auto two = [&](uint32_t b) {
            return half2_of(scale_exp2(__uint_as_float(b << 16), ex), scale_exp2(__uint_as_float(b & 0xFFFF0000u), ex));
          };
          *reinterpret_cast<uint4*>(sh.q[i] + tile_chunk(c >> 3, row, c & 7)) =
              make_uint4(two(x.x), two(x.y), two(x.z), two(x.w));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.q_full[i]);

        // ---- limits of this row and of the row tile
        // not zero: a masked score is -Inf before it is multiplied
        float factor = fmaxf(scale_exp2(a.scale * kg * kLog2e, kValueExp - ex), 1.17549435e-38f);
        const bool of_row = factor > kHugeFactor<D>, huge = __any_sync(0xFFFFFFFFu, of_row);
        if (huge) sh.factor[tid] = of_row ? factor : 1.0f;  // a row's scores are multiplied before the maximum, not with it
        if (of_row) factor = 1.0f;
        const int64_t pos0 = (int64_t)w.seq.len - w.seq.rows;
        const int32_t r_last = (nrows - r0 < 128 ? nrows : r0 + 128) - 1;
        const Visible first_row = visible(pos0 + a.by_group.divide(r0), w.seq.len, a.causal, a.window);
        const Visible last_row = visible(pos0 + a.by_group.divide(r_last), w.seq.len, a.causal, a.window);
        Visible mine = visible(pos0 + t, w.seq.len, a.causal, a.window);
        if (!live) mine = Visible{0, 0x7FFFFFFF};  // never written
        // lanes 0..3: the pages of the next step's granules (0 behind the span), looked at one step later
        const int32_t* table = a.ix.table + (int64_t)w.b * a.ix.width;
        const int32_t gend = w.span.g0 + w.span.n;
        int32_t gi = w.span.g0 + kUnitGranules * j0 + (lane & 3);
        auto page_at = [&](int32_t g) {
          return g < gend && NVFP4_IN_BOUNDS(g >> a.ix.gshift, a.ix.width, a.status) ? table[g >> a.ix.gshift] : 0;
        };
        int32_t page = page_at(gi);
        int32_t tok0 = (w.span.g0 + kUnitGranules * j0) * kGranule;
        const int32_t all_lo = last_row.lo, all_hi = w.span.n > 0 ? first_row.hi : 0;

        float m = kStartMax, l = 0.0f;
        for (int x = 2 * (j1 - j0); x > 0; --x, ++steps, tok0 += 64) {
          const uint32_t bad = __ballot_sync(0xFFFFFFFFu, page < 0 || page >= a.ix.num_pages);
          gi += 4;
          page = page_at(gi);
          const bool whole = tok0 >= all_lo && tok0 + 64 <= all_hi && bad == 0;
          const uint32_t t_x = t_s + 64 * (steps & 1);
          if (!(ok = wait(&sh.s_full[i][steps & 1], (steps >> 1) & 1))) break;
          tc_fence_after();
          if (!whole) {  // what a row does not see becomes -Inf in place
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              uint32_t y[16];
              tmem_read16(t_x + 16 * c, y);
              const int32_t t0 = tok0 + 16 * c;
              const bool none = (bad >> c) & 1u;
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if (none || t0 + e < mine.lo || t0 + e >= mine.hi) y[e] = 0xFF800000u;
              tmem_st16(t_x + 16 * c, y);
            }
            tmem_wait_st();
          }
          uint32_t y[64];
          tmem_read64(t_x, y);
          if (huge) {
            const float f = sh.factor[tid];
#pragma unroll
            for (int e = 0; e < 64; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * f);
          }
          float t0 = -INFINITY, t1 = t0, t2 = t0, t3 = t0;
#pragma unroll
          for (int e = 0; e < 64; e += 8) {
            t0 = max3_nan(t0, __uint_as_float(y[e]), __uint_as_float(y[e + 1]));
            t1 = max3_nan(t1, __uint_as_float(y[e + 2]), __uint_as_float(y[e + 3]));
            t2 = max3_nan(t2, __uint_as_float(y[e + 4]), __uint_as_float(y[e + 5]));
            t3 = max3_nan(t3, __uint_as_float(y[e + 6]), __uint_as_float(y[e + 7]));
          }
          const float top = max3_nan(max2_nan(t0, t1), t2, t3) * factor;
          if (__any_sync(0xFFFFFFFFu, !(top - m <= kRescaleAt + kHeadroom))) {
            // (a score of NaN or +Inf stays in m: the sum would not show it where exp2_poly has its place)
            const float m1 = top < INFINITY ? new_max(top, m) : NAN;
            const float f = m == kStartMax ? 0.0f : ex2(m - m1);
            m = m1;
            l *= f;
            if (x < 2 * (j1 - j0)) {
              // O at rest. (The buffer's earlier P V is known to be complete, or its S could not have come: the parity is
              // not ambiguous.)
              if (!(ok = wait(&sh.pv_done[i][(steps - 1) & 1], ((steps - 1) >> 1) & 1))) break;
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < D / 16; ++c) {
                uint32_t o[16];
                tmem_read16(t_o + 16 * c, o);
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tmem_st16(t_o + 16 * c, o);
              }
            }
          }
          // p as FP16 pairs (to 2^-11 of itself from 2^-14 on, below to 2^-25) into the first half of the buffer
          f32x2 sum = 0;
          const f32x2 ff = pack2(factor, factor), mm = pack2(-m, -m);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t p[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float a0, a1;
              const f32x2 z =
                  fma2(pack2(__uint_as_float(y[32 * c + 2 * e]), __uint_as_float(y[32 * c + 2 * e + 1])), ff, mm);
              if (e % kPolyEvery == kPolyEvery - 1) {
                exp2_poly(z, a0, a1);
              } else {
                unpack2(z, a0, a1);
                a0 = ex2(a0);
                a1 = ex2(a1);
              }
              sum = add2(sum, pack2(a0, a1));
              p[e] = half2_of(a0, a1);
            }
            tmem_st16(t_x + 16 * c, p);
          }
          {
            float s0, s1;
            unpack2(sum, s0, s1);
            l += s0 + s1;
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.p_full[i][steps & 1]);
        }
        if (!ok) break;

        // ---- epilogue: O of the last step is complete
        if (!(ok = wait(&sh.pv_done[i][(steps - 1) & 1], ((steps - 1) >> 1) & 1))) break;
        tc_fence_after();
        const bool whole_work = from_unit() == 0 && to_unit() == w.n;
        const int64_t at = tok * a.ix.hkv * a.group + hq;
        if (m == kStartMax) m = -INFINITY;
        auto write_row = [&](int c, const float* o, float f) {  // 32 dimensions from 32*c
          uint4* out = reinterpret_cast<uint4*>(a.out + at * D + 32 * c);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float* x = o + 8 * e;
            out[e] = make_uint4(f32x2_to_bf16x2(x[0] * f, x[1] * f), f32x2_to_bf16x2(x[2] * f, x[3] * f),
                                f32x2_to_bf16x2(x[4] * f, x[5] * f), f32x2_to_bf16x2(x[6] * f, x[7] * f));
          }
        };
        const bool write = live && NVFP4_IN_BOUNDS(at, a.ix.total * a.ix.hkv * a.group, a.status);
        if (whole_work) {
          // (by the maximum: l of a row that saw nothing holds the 2^-126 that exp2_poly gives for a masked score)
          const float f = m == -INFINITY ? 0.0f : output_factor(vg, l);
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_read32(t_o + 32 * c, o);
            if (write) write_row(c, reinterpret_cast<const float*>(o), f);
          }
          if (write && a.lse) a.lse[at] = m == -INFINITY ? -INFINITY : (m + log2f(l)) * kLn2;
        } else {
          // part of a work: m, l, then O in pieces of 4 columns x 128 rows
          constexpr int kPart = 128 * (D + 2);
          auto part_of = [&](int64_t cta, bool head_part) { return a.partial + ((2 * cta + head_part) * 2 + i) * kPart; };
          float* mine_p = part_of(blockIdx.x, from_unit() == 0);
          mine_p[row] = m;
          mine_p[128 + row] = l;
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_read32(t_o + 32 * c, o);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              *reinterpret_cast<uint4*>(mine_p + 256 + ((8 * c + e) * 128 + row) * 4) =
                  make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
          if (!(ok = meet())) break;
          const int64_t c0 = w.w0 / sh.part.per, c1 = (w.w0 + w.n - 1) / sh.part.per;
          if (row == 0) sh.last[i] = arrive_last(a.counters + 2 * c0 + i, (int)(c1 - c0));
          if (!(ok = meet())) break;
          if (sh.last[i]) {
            float mt = -INFINITY, lt = 0.0f;
            for (int64_t c = c0; c <= c1; ++c) mt = max2_nan(mt, __ldcg(part_of(c, c == c0) + row));
            for (int64_t c = c0; c <= c1; ++c) {
              const float mc = __ldcg(part_of(c, c == c0) + row);
              lt += mc == -INFINITY ? 0.0f : __ldcg(part_of(c, c == c0) + 128 + row) * ex2(mc - mt);
            }
            const float f = lt == 0.0f ? 0.0f : output_factor(vg, lt);
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              float o[32];
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = 0.0f;
              for (int64_t x = c0; x <= c1; ++x) {
                const float* from = part_of(x, x == c0);
                const float mc = __ldcg(from + row);
                const float g = mc == -INFINITY ? 0.0f : ex2(mc - mt);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  const float4 y = __ldcg(reinterpret_cast<const float4*>(from + 256 + ((8 * c + e) * 128 + row) * 4));
                  o[4 * e] += y.x * g;
                  o[4 * e + 1] += y.y * g;
                  o[4 * e + 2] += y.z * g;
                  o[4 * e + 3] += y.w * g;
                }
              }
              if (write) write_row(c, o, f);
            }
            if (write && a.lse) a.lse[at] = lt == 0.0f ? -INFINITY : (mt + log2f(lt)) * kLn2;
          }
          if (!(ok = meet())) break;  // sh.last is read before the next work writes it
        }
        tc_fence_before();
      }
      if (!next_work()) break;
    }
    if (!ok) timed_out();
  } else if (warp < 12) {
    // ------------------------------------------------------ dequantization
    const int dw = warp - 8;
    uint32_t it = 0;  // K/V tiles done
    bool ok = true;
    while (ok) {
      int j0, j1;
      tiles_of_part(j0, j1);
      for (int x = j1 - j0; x > 0; --x, ++it) {
        const uint32_t st = it % kStages;
        if (!(ok = wait(&sh.codes_full[st], (it / kStages) & 1))) break;
        const uint32_t there = uniform((int)sh.there[st]);
#pragma unroll
        for (uint32_t which = 0; which < 2; ++which) {
          // K or V of granules dw and dw + 4 into rows 16*dw.. and 64 + 16*dw.. of an FP16 tile, zeros for those that
          // are not there; two lanes share the 64 dimensions of half h of a token. All loads come first: the stores
          // may not be moved behind them, and each trip would wait for shared memory twice.
          uint4 codes[2][D / 64];
          uint32_t sc[2][D / 64];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint8_t* gr = sh.codes[st][dw + 4 * y] + which * 9 * D;
            const bool some = (there >> (dw + 4 * y)) & 1u;
#pragma unroll
            for (int h = 0; h < D / 64; ++h) {
              codes[y][h] = make_uint4(0, 0, 0, 0);
              sc[y][h] = 0;
              if (some) {
                codes[y][h] = *reinterpret_cast<const uint4*>(gr + (lane >> 1) * (D / 2) + h * 32 + (lane & 1) * 16);
                sc[y][h] =
                    *reinterpret_cast<const uint16_t*>(gr + 8 * D + (lane >> 1) * (D / 16) + h * 4 + (lane & 1) * 2);
              }
            }
          }
          const uint32_t tile = 2 * it + which;
          if (!(ok = wait(&sh.empty[place(tile)], turn_of(tile) ^ 1))) break;
          uint8_t* to = sh.kv[place(tile)];
#pragma unroll
          for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int h = 0; h < D / 64; ++h) {
              const uint32_t cw[4] = {codes[y][h].x, codes[y][h].y, codes[y][h].z, codes[y][h].w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint32_t f = scales_to_half(__byte_perm(sc[y][h], 0, e < 2 ? 0x4040 : 0x4141));
                uint32_t o[4];
                codes_to_half(cw[e], o);
                *reinterpret_cast<uint4*>(
                    to + tile_chunk(h, (dw + 4 * y) * kGranule + (lane >> 1), (lane & 1) * 4 + e)) =
                    make_uint4(hmul2(o[0], f), hmul2(o[1], f), hmul2(o[2], f), hmul2(o[3], f));
              }
            }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.full[place(tile)]);
        }
        if (!ok) break;
        if (lane == 0) mbar_arrive(&sh.codes_empty[st]);
      }
      if (!ok || !next_work()) break;
    }
    if (!ok) timed_out();
  } else if (warp == 14) {
    // ------------------------------------------- bulk copies of the codes
    uint32_t it = 0;
    bool ok = true;
    while (ok) {
      int j0, j1;
      tiles_of_part(j0, j1);
      const int n = j1 - j0;
      const int32_t* table = a.ix.table + (int64_t)w.b * a.ix.width;
      const int32_t gend = w.span.g0 + w.span.n;
      const int64_t page_bytes = ((int64_t)a.ix.hkv << a.ix.gshift) * kGB;
      const uint8_t* head = a.pages + ((int64_t)w.head << a.ix.gshift) * kGB;
      int32_t gi = w.span.g0 + kUnitGranules * j0 + (lane & 7);  // lanes 0..7: a granule each
      auto page_of = [&](int32_t g) {  // -2 behind the span
        return g < gend && NVFP4_IN_BOUNDS(g >> a.ix.gshift, a.ix.width, a.status) ? table[g >> a.ix.gshift] : -2;
      };
      int32_t page = page_of(gi);
      for (int x = 0; x < n; ++x, ++it, gi += kUnitGranules) {
        const uint32_t st = it % kStages;
        const int32_t next = page_of(gi + kUnitGranules);
        const bool good = page >= 0 && page < a.ix.num_pages;
        if (!good && page != -2) record_status(a.status, NVFP4_ERR_PAGE);
        int64_t at = page * page_bytes + (int64_t)(gi & ((1 << a.ix.gshift) - 1)) * kGB;
        if (good && !NVFP4_IN_BOUNDS(at + kGB - 1, a.ix.num_pages * page_bytes, a.status)) at = 0;
        const uint32_t there = __ballot_sync(0xFFFFFFFFu, good) & 0xFFu;
        if (!(ok = wait(&sh.codes_empty[st], ((it / kStages) & 1) ^ 1))) break;
        if (lane == 0) {
          sh.there[st] = there;
          mbar_arrive_expect_tx(&sh.codes_full[st], (uint32_t)__popc(there) * kGB);
        }
        __syncwarp();
        if (lane < 8 && good && it >= (uint32_t)a.withheld) bulk_load(sh.codes[st][lane], head + at, kGB, &sh.codes_full[st]);
        page = next;
      }
      if (!ok || !next_work()) break;
    }
    if (!ok) timed_out();
    // the last tiles' copies land, even if those who wait for them gave up
    for (uint32_t x = it < kStages ? 0 : it - kStages; x < it; ++x) settle(&sh.codes_full[x % kStages], (x / kStages) & 1);
    __syncwarp();
  } else {
    // ----------------------------------------------------------- MMA issue
    if (warp < 14) {
      const int i = warp - 12;
      constexpr uint32_t idesc_s = idesc_f16(64, false), idesc_o = idesc_f16(D, true);
      const uint32_t t_s = tmem + i * 128, t_o = tmem + 256 + i * D;
      uint32_t it = 0, steps = 0, works = 0;
      bool ok = true;
      const uint64_t qd = smem_desc(smem_u32(sh.q[i]), 16, 1024, 2);
      auto scores = [&](uint32_t t, uint32_t half) {  // S = Q K^T of 64 tokens (64 rows of 128 bytes) of tile t
        const uint32_t st = place(2 * t);
        if (half == 0) {
          if (!wait(&sh.full[st], turn_of(2 * t))) return false;
          tc_fence_after();
        }
        mma_scores<D>(t_s + 64 * half, qd, smem_desc(smem_u32(sh.kv[st]), 16, 1024, 2) + half * 512, idesc_s);
        tc_commit_elect(&sh.s_full[i][half]);
        if (half) tc_commit_elect(&sh.empty[st]);
        return true;
      };
      while (ok) {
        int j0, j1;
        tiles_of_part(j0, j1);
        const int n = j1 - j0;
        if (w.tile * kPreRows + i * 128 < w.seq.rows * a.group) {
          if (!(ok = wait(&sh.q_full[i], works & 1))) break;
          ++works;
          tc_fence_after();
          if (!(ok = scores(it, 0) && scores(it, 1))) break;
          for (int j = 0; j < n; ++j, ++it) {
            const uint32_t st = place(2 * it + 1);
            if (!(ok = wait(&sh.full[st], turn_of(2 * it + 1)))) break;
            const uint64_t vd = smem_desc(smem_u32(sh.kv[st]), kTileTokens * 128, 1024, 2);
#pragma unroll
            for (uint32_t half = 0; half < 2; ++half, ++steps) {
              if (!(ok = wait(&sh.p_full[i][half], (steps >> 1) & 1))) break;
              tc_fence_after();
              mma_values(t_o, t_s + 64 * half, vd + half * (4 * 2048 / 16), idesc_o, (j | (int)half) != 0);
              tc_commit_elect(&sh.pv_done[i][half]);
              if (half) tc_commit_elect(&sh.empty[st]);
              if (!(ok = wait(&sh.pv_done[i][half], (steps >> 1) & 1))) break;
              if (j + 1 < n && !(ok = scores(it + 1, half))) break;
            }
            if (!ok) break;
          }
        } else {  // no rows in this half: the stages are only passed on
          for (int j = 0; j < n && ok; ++j, ++it) {
            for (uint32_t tile = 2 * it; ok && tile < 2 * it + 2; ++tile) {
              ok = wait(&sh.full[place(tile)], turn_of(tile));
              if (ok && lane == 0) mbar_arrive(&sh.empty[place(tile)]);
            }
            __syncwarp();
          }
        }
        if (!ok || !next_work()) break;
      }
      if (!ok) {
        timed_out();
        tc_commit_elect(&sh.drain[i]);  // MMAs in flight read shared memory
        settle(&sh.drain[i], 0);
      }
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

constexpr int kMaxPreCtas = 160;

size_t kv_prefill_partial_floats() { return (size_t)kMaxPreCtas * 4 * 128 * (128 + 2); }

template <int D>
cudaError_t launch_tiles(AttnArgs a, int num_sms, cudaStream_t s) {
  constexpr int bytes = (int)sizeof(PreShared<D>) + 1024;
  static_assert(bytes <= 232448, "shared memory budget");
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void*>(&kv_prefill_kernel<D>), bytes, done);
  if (e != cudaSuccess) return e;
  const int grid = num_sms < kMaxPreCtas ? num_sms : kMaxPreCtas;
  a.by_grid = Divisor(grid);
  note_launch();
  kv_prefill_kernel<D><<<grid, kPreThreads, bytes, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_kv_prefill(const AttnArgs& a, int D, int num_sms, cudaStream_t s) {
  return D == 128 ? launch_tiles<128>(a, num_sms, s) : launch_tiles<64>(a, num_sms, s);
}

}  // namespace nvfp4
