// Split-KV attention over E4M3 pages with one scale per (page, kv head), on
// fp8 tensor-core operands (tcgen05 kind::f8f6f4): the codes go from the page
// to the MMA as they are.
//
// For one (request b, kv head h) with R = G*K packed query rows (r = i*G + g)
// and keys j at logical position j, page slot j / P:
//   x_rj = sum_d q_rd kc_jd          (kc, vc: the stored codes)
//   s_rj = scale log2(e) ks_j x_rj   (ks, vs: the page's scales)
//   lse2_r = log2 sum_j 2^s_rj,      out_r = sum_j 2^(s_rj - lse2_r) vs_j vc_j.
// With ws_j = vs_j / vs_0 (vs_0: the scale of the unit's first page),
// t_rj = s_rj + log2(ws_j) and a bias n_r per row such that t_rj + n_r <= 8 the
// sums the kernel keeps are
//   O_rd = sum_j P_rj vc_jd,  l_r = sum_j P_rj / ws_j,  P_rj = 2^(t_rj + n_r),
// so out = vs_0 O / l and lse2 = log2(l) - n: the value scale rides in the
// exponent and costs no product per key.  Taken relative to vs_0, a cache whose
// scales are all near 2^-100 (values of zero) stays in the middle of fp32's
// range.  ws_j is held at 2^-64 or more: a page that quiet adds nothing to sums
// that the first one's scale is part of, and 1 / ws_j cannot overflow l.  Upwards
// it may reach 2^100: keys 2^-32 of a row's largest are still in l.
//
// bf16 factors on fp8 operands.  A bf16 value has 8 significant bits, an E4M3
// code 4: q (times one power of two per tile, which puts the tile's largest
// magnitude in [2^7, 2^8)) is hi + lo with both terms E4M3, exactly down to
// 2^-10 of the largest value and to 2^-18 of it below; both terms accumulate
// into the same scores.  Rows far below the loudest (a quiet head, or all others
// beside a padding token of any size) would lose theirs: where the largest
// elements of rows lie more than kP8Apart powers of two apart, the unit is taken
// again for the quieter ones, under their own power, until none is left.  (At a
// distance g the scores of a row are off by about 2^(g - 18) of their deviation,
// so at 6 by 2^-12.  The further pass costs a unit's whole time again, and every
// other call 0 to 3 %: 64/4 window 102.5 -> 105.8 us.  A power for each row within
// one pass: 107.8.)
//
// P is hi + lo / 32: hi is P rounded to 4 bits, lo the rest times 32, rounded to 4
// bits, so P keeps a relative 2^-8.7 (with its step through f16) down to 2^-6,
// and 2^-15 below; the two terms accumulate apart and join in the epilogue.  Only
// the tile at hand has to fit that range: O and l are fp32 and are rescaled when
// the bias moves, down for a key louder than all before and up again for the tail
// behind it, which would otherwise flush to zero (with 131072 keys behind one of
// 0.9 of the weight and a value of zero, all of the output; now 0.2 % of it).
// What stays lost are keys that share a tile with a far louder one: below 2^-23
// of it where it stands alone, else 2^-19, so at most 127 times that of a row's
// weight each time.
//
// Transposed products, keys along M:
//   S^T [128 keys x RP rows] = K [128 x D] (K-major, as TMA lands it) Q^T,
//   O^T [D x 2 RP] += V^T (MN-major, as TMA lands it) [P_hi | P_lo],
// so a shape with few query rows wastes nothing: the MMA's M is 128 keys or
// the D columns of V, its N the rows.  A softmax thread owns one key (its
// TMEM lane) and RP / NG rows: the scales are per-thread scalars, the mask is
// a row interval, and P goes to shared memory as 16-byte pieces.  What the
// threads of a row must share is the bias n_r: it is set from the row's
// largest t in its first tile (to P = 2^4, which leaves scores four bits to
// grow) and moves when a P would pass 2^8, which the group's four warps agree
// on by one barrier per tile that also carries the vote, or when a look at the
// tile's column maxima (the second tile, every 16th, and the one behind a large
// step down) finds a row below 2^-5.
//
// Grid (splits, Hkv, B), one unit of C 128-key tiles per CTA, as the mma.sync
// kernel; the combine kernel merges the units.
// Warps: 4 TG NG softmax warps, then the K producer, the V producer, the QK^T
// issuer and the PV issuer.  A tile's softmax is a chain (score load, vote,
// exponentials, stores, fence) of 1400 to 2600 cycles, against the 700
// (D = 64) or 1400 (D = 128) that its codes take from HBM, so tiles have to
// overlap: up to 32 rows by two or three CTAs on an SM, at 48 and 64 by TG = 2
// tile groups of four warps (quadrant = warp % 4) that take tiles tg, tg + TG,
// ... with biases, sums and an O accumulator of their own, joined at the end;
// above, where tensor memory has room for one accumulator, two row groups
// share a tile and only the products overlap the softmax.
// A producer keeps the page ids of the next 32 page slots in its lanes, and
// each lane issues its own page's box; the K producer also puts each tile's
// page scales into a ring.  Every mbarrier wait is bounded; a warp whose wait
// ran out goes on with whatever it finds up to its group's next vote, where
// the group stops.
//
// Measured, replayed in a CUDA graph (bytes: codes, scales, tables and rows over
// 6.77 TB/s, the rate of a plain copy): 24 requests of 1K to 128K keys, 64/16
// heads of 64, 7 tokens 608 us, 77 % of that rate; 32 x 128K keys, 12/2 heads of
// 64, 7 tokens 277 us, 57 %; 64 requests with a window of 4096, 7 tokens, 64/4
// heads of 128 103 us, 41 %; 48 requests of 1 to 9001 keys, 8/2 heads of 64,
// single tokens 21 us, 39 %.  From 48 rows on the chain bounds it, not the bytes:
// two or three warps a scheduler issue in two thirds of the cycles, and a unit
// pays 7 to 12 us before its first and behind its last full-speed tile (112 rows
// of 128 10.5; up to 32 rows 4 to 7, shared by the CTAs of an SM).

#include <cuda_runtime.h>

#include "device_common.cuh"
#include "tcgen05.cuh"

namespace dflash {
namespace {

constexpr int kP8T = 128;                // keys per tile
// A row's bias.  When it is first set and when it moves, its tile's largest P is
// put to 2^kP8Set, or to 2^kP8Limit where that of 32 keys lies kP8Alone above
// those of the other 96, in the first tile or with a step as large (a key that
// stands alone is not soon passed, and what shares its tile keeps four bits
// more).  A P past 2^kP8Limit moves it, and with it every row of the group above
// 2^kP8Off.  Looks (the second tile, every kP8Every-th but the last few, the one
// behind a step down of kP8Drop or more) move rows whose tile stays below
// 2^kP8Low, but never more than kP8Rise above the lowest bias the row had: 2^17
// keys 2^-32 below the loudest weigh 2^-15 of it.
// Measured, 64/4 heads of 128 with a window of 4096 / 12/2 heads of 64 at 128K, 7
// tokens, scores of deviation 1 (and 3): only falling, first at 2^3, 98 (125) /
// 268 (303) us, but the tail lost; these values 103 (138) / 274 (358).  A look
// every 32nd tile 102 / 272, every 8th 105 / 275; kP8Drop at -8 (148) / (390);
// only rows past 2^kP8Limit moved 117 / 283.
constexpr float kP8Limit = 8.f;
constexpr float kP8Set = 4.f;
constexpr float kP8Off = 4.5f;
constexpr float kP8Alone = 6.f;
constexpr float kP8Low = -5.f;
constexpr float kP8Rise = 32.f;
constexpr float kP8Drop = -10.f;
constexpr int kP8Every = 16;
constexpr float kP8Quietest = -64.f;     // least log2 of a value scale over the first page's
enum : uint8_t { kRowTaken, kRowPutOff, kRowDone };  // of a pass over the unit
constexpr uint32_t kP8Apart = 6;         // powers of two between the largest queries of rows taken together

// Tile and row groups, CTAs per SM and ring stages by head dim and padded rows.
// Measured, one side against the other, inputs not in L2:
//   CTAs per SM, 16 rows: 3 / 2 / 1 at D = 64 25.4 / 26.4 / 38.2 us, 2 / 1 at
//   D = 128 30.0 / 40.2 (48 requests of 1 to 9001 keys, 8/2 heads; at D = 128
//   shared memory ends at 2).
//   32 rows: 2 / 1 351 / 522 us at D = 64 (24 requests of 1K to 64K keys, 64/16
//   heads, 7 tokens), 278 / 329 at D = 128 (to 32K); two to four tile groups in
//   one CTA instead were slower, too.
//   Tile groups, 48 rows: 2 / 1 281 / 377 us (D = 64, 32 x 128K keys, 12/2
//   heads, 7 tokens); three have no registers left and were slower.  64 rows:
//   2 / 1 77 / 84 us at D = 128, 71 / 81 at D = 64 (64 requests, window 4096,
//   64/4 heads, 4 tokens).
//   Above 64 rows a thread holds its scores and sums of RP / 2 rows: more do
//   not fit its registers, nor a second accumulator the tensor memory.
template <int D, int RP>
struct P8Cfg {
  static constexpr int TG = RP == 48 || RP == 64 ? 2 : 1;        // tile groups
  static constexpr int NG = RP > 64 ? 2 : 1;                     // row groups
  static constexpr int NR = RP / NG;                             // rows per softmax thread
  static constexpr int NB = 2 * TG;                              // S and P buffers, two per tile group: tile j has j % NB
  static constexpr int kCtas = RP <= 16 ? (D == 64 ? 3 : 2) : (RP <= 32 ? 2 : 1);
  static constexpr int NSK = D == 64 ? (RP <= 16 ? 3 : (RP <= 32 ? 4 : (RP <= 48 ? 9 : 6))) : (RP <= 32 ? 3 : 4);
  static constexpr int NSV = D == 64 ? (RP <= 16 ? 3 : (RP <= 32 ? 4 : (RP <= 48 ? 9 : 6))) : (RP <= 32 ? 2 : (RP <= 64 ? 4 : 3));
  static constexpr int kSoftWarps = 4 * TG * NG;
  static constexpr int kThreads = 32 * (kSoftWarps + 4);
  static constexpr int kTile = kP8T * D;                  // codes of one K or V tile
  static constexpr int kQ = RP * D;                       // one term of the query tile
  // P: hi and lo of every row are 2 RP columns, kPRow bytes of a key to a
  // block; two row groups of more than 16 rows have a block each, so that a
  // thread's pieces lie one XOR apart.
  static constexpr bool kOwnBlock = NG == 2 && NR > 16;
  static constexpr int kPRow = RP <= 32 ? 64 : 128;
  static constexpr int kPBlock = kP8T * kPRow;
  static constexpr int kP = (kOwnBlock ? 2 : 1) * kPBlock;  // one P buffer
  static constexpr int kPCols = kOwnBlock ? 128 + 2 * NR : 2 * RP;
  static constexpr int kRing = NSK + NB;                  // page-scale entries, by tile
  static constexpr int kOffQ = 0;
  static constexpr int kOffP = 2 * kQ;
  static constexpr int kOffK = kOffP + NB * kP;
  static constexpr int kOffV = kOffK + NSK * kTile;
  static constexpr int kOffBar = kOffV + NSV * kTile;
  // k_full, k_empty, v_full, v_empty, scales, s_full, s_free, p_full, pv_done, q_full
  static constexpr int kNumBars = 2 * NSK + 2 * NSV + kRing + 4 * NB + 1;
  static constexpr int kOffMisc = kOffBar + (kNumBars * 8 + 15) / 16 * 16;
  static constexpr int kOffScale = kOffMisc + 64;              // float4 [kRing][8]
  static constexpr int kOffRow = kOffScale + kRing * 8 * 16;
  // float [TG][RP] each: bias, cap, delta, fac; then colmax [TG][4][RP]
  static constexpr int kOffState = kOffRow + 8 * TG * RP * 4;  // uint8 [RP]
  static constexpr int kSmem = kOffState + RP + 1024;
  static constexpr int kColO = NB * RP;  // tensor memory: NB score buffers of RP columns, TG accumulators of kPCols
  static constexpr int kCols = kColO + TG * kPCols;
  static constexpr int kTmem = kCols <= 64 ? 64 : (kCols <= 128 ? 128 : (kCols <= 256 ? 256 : 512));
  static_assert(RP % 16 == 0 && NR % 8 == 0 && NR * NG == RP, "rows");
  static_assert(kSmem <= 232448 && kCtas * (kSmem + 1024) <= 228 * 1024, "shared memory");
  static_assert(kCols <= 512 && kCtas * kTmem <= 512, "tensor memory");
  static_assert(kOffP % 1024 == 0 && kOffK % 1024 == 0 && kTile % 1024 == 0, "tile alignment");
};

__device__ __forceinline__ float p8_ninf() { return __int_as_float(0xff800000); }

__device__ __forceinline__ float redux_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// Barrier over `count` threads that also gives each whether any came with p.
__device__ __forceinline__ bool barrier_any(int id, int count, bool p) {
  int any;
  asm volatile(
      "{\n\t.reg .pred a, b;\n\tsetp.ne.s32 a, %1, 0;\n\t"
      "barrier.cta.red.or.pred b, %2, %3, a;\n\tselp.s32 %0, 1, 0, b;\n\t}"
      : "=r"(any)
      : "r"(p ? 1 : 0), "r"(id), "r"(count)
      : "memory");
  return any != 0;
}

__device__ __forceinline__ void mbar_inval(uint32_t bar) {
  asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// mbar_wait_warp, cheaper where the phase has usually completed.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return mbar_wait_warp(bar, parity);
}

template <int N>
__device__ __forceinline__ void load_scores(uint32_t taddr, uint32_t (&r)[N]) {
  static_assert(N == 16 || N == 32 || N == 48 || N == 56 || N == 64, "score columns");
  if constexpr (N == 16) tmem_ld16_wait(taddr, r);
  else if constexpr (N == 32) tmem_ld32_wait(taddr, r);
  else if constexpr (N == 48) tmem_ld48_wait(taddr, r);
  else if constexpr (N == 56) tmem_ld56_wait(taddr, r);
  else tmem_ld64_wait(taddr, r);
}

// d = a * b + c, two at a time.
__device__ __forceinline__ void fma2(float& d0, float& d1, float a0, float a1, float b, float c0, float c1) {
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %4};\n\tmov.b64 c, {%5, %6};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b), "f"(c0), "f"(c1));
}

// a + c, b + c.
__device__ __forceinline__ void add2(float& a, float& b, float c) {
  asm("{\n\t.reg .b64 a, c;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 c, {%2, %2};\n\t"
      "add.rn.f32x2 a, a, c;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(c));
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Sums of 8 values over the warp's lanes: lane L returns that of value L / 4,
// by halving (each step a lane keeps half of its values).
__device__ __forceinline__ float sum8(float (&v)[8], int lane) {
#pragma unroll
  for (int step = 0; step < 3; ++step) {
    const int half = 4 >> step, m = 16 >> step;
    const bool up = (lane & m) != 0;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float keep = up ? v[i + half] : v[i];
      const float send = up ? v[i] : v[i + half];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, m);
    }
  }
  const float w = v[0] + __shfl_xor_sync(0xffffffffu, v[0], 2);
  return w + __shfl_xor_sync(0xffffffffu, w, 1);
}

// P of four rows of a key -> one word of hi codes and one of lo codes.
// f16 holds P <= 2^8 with 11 bits; hi is its nearest E4M3 value, and
// 32 (P - hi) is exact in f16 and at most 2^8.  (P as one f16 operand, with the
// value codes widened to f16 in shared memory, saves these conversions, but the
// widening lengthens the chain: 8 % at 112 rows, 119 us against 110 when that was
// this form's time.)
__device__ __forceinline__ void split_p4(float p0, float p1, float p2, float p3, uint32_t& hi, uint32_t& lo) {
  const uint32_t h01 = pack_f16x2(p0, p1), h23 = pack_f16x2(p2, p3);
  asm("{\n\t.reg .b16 a, b, c, d;\n\t.reg .b32 x, y, u, v, k, n;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 a, %2;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 b, %3;\n\t"
      "mov.b32 %0, {a, b};\n\t"
      "cvt.rn.f16x2.e4m3x2 x, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 y, b;\n\t"
      "mov.b32 k, 0x50005000;\n\t"   // 32.0 in both halves
      "mov.b32 n, 0xD000D000;\n\t"   // -32.0
      "mul.rn.f16x2 u, %2, k;\n\t"
      "mul.rn.f16x2 v, %3, k;\n\t"
      "fma.rn.f16x2 u, x, n, u;\n\t"
      "fma.rn.f16x2 v, y, n, v;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 c, u;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 d, v;\n\t"
      "mov.b32 %1, {c, d};\n\t}"
      : "=r"(hi), "=r"(lo)
      : "r"(h01), "r"(h23));
}

// Two query values (times qs) -> their hi and lo E4M3 codes, first value in
// the low byte.  A value that is not finite becomes the NaN code.
__device__ __forceinline__ void split_q2(float a, float b, uint32_t& hi, uint32_t& lo) {
  uint16_t h, l;
  const float nan = __int_as_float(0x7fffffff);
  a = fabsf(a) <= 3.4028235e38f ? a : nan;
  b = fabsf(b) <= 3.4028235e38f ? b : nan;
  uint32_t back;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(b), "f"(a));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(back) : "h"(h));
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&back));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(l) : "f"(b - f.y), "f"(a - f.x));
  hi = h;
  lo = l;
}

// One pass of a CTA over its unit, for the query rows that lie near the loudest
// of those not yet done.  Returns whether rows are left for another pass (alike
// in every thread).  RERUN: not the first.
template <int D, int RP, bool RERUN>
__device__ __forceinline__ bool unit_pass(const AttnArgs& a, const float* __restrict__ k_scales, const float* __restrict__ v_scales,
                                          const CUtensorMap& tm_k, const CUtensorMap& tm_v) {
  using C = P8Cfg<D, RP>;
  constexpr int T = kP8T;
  constexpr int NR = C::NR;
  constexpr int TG = C::TG;
  constexpr int NG = C::NG;
  constexpr int NB = C::NB;
  constexpr int kSoft = 32 * C::kSoftWarps;  // softmax threads
  constexpr int NSK = C::NSK;
  constexpr int NSV = C::NSV;

  const int s = blockIdx.x;
  const int h = blockIdx.y;
  const int b = blockIdx.z;
  const int L_raw = __ldg(&a.ctx_lens[b]);
  const Geometry geo = make_geometry(L_raw, a.max_ctx_len, a.K, a.W, T, a.C);
  if (!RERUN && threadIdx.x == 0 && s == 0 && h == 0 && (L_raw < 0 || L_raw > a.max_ctx_len))
    flag_status(a.status, DFLASH_STATUS_BAD_CTX_LEN);
  if (s >= geo.n_splits) return false;  // empty split unit (uniform over the CTA)
  const int tile0 = geo.t_begin + s * a.C;
  const int n = min(geo.n_tiles - s * a.C, a.C);

  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_u32 = smem_u32(smem_raw);
  const uint32_t base = (raw_u32 + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw_u32);
  const uint32_t bars = base + C::kOffBar;
  auto k_full = [&](int st) { return bars + 8u * st; };
  auto k_empty = [&](int st) { return bars + 8u * (NSK + st); };
  auto v_full = [&](int st) { return bars + 8u * (2 * NSK + st); };
  auto v_empty = [&](int st) { return bars + 8u * (2 * NSK + NSV + st); };
  constexpr int kB0 = 2 * NSK + 2 * NSV;
  auto scales_full = [&](int e) { return bars + 8u * (kB0 + e); };
  constexpr int kB1 = kB0 + C::kRing;
  auto s_full = [&](int p) { return bars + 8u * (kB1 + p); };
  auto s_free = [&](int p) { return bars + 8u * (kB1 + NB + p); };
  auto p_full = [&](int p) { return bars + 8u * (kB1 + 2 * NB + p); };
  auto pv_done = [&](int p) { return bars + 8u * (kB1 + 3 * NB + p); };
  const uint32_t q_full = bars + 8u * (kB1 + 4 * NB);
  uint32_t* misc = reinterpret_cast<uint32_t*>(gbase + C::kOffMisc);
  volatile uint32_t* tmem_slot = misc;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
  volatile int* issued_k = reinterpret_cast<volatile int*>(misc + 2);
  volatile int* issued_v = reinterpret_cast<volatile int*>(misc + 3);
  uint32_t* q_amax = misc + 4;                                            // largest |q| of the rows taken, as bits
  volatile uint32_t* q_rest = misc + 5;                                   // 1: some rows lie far below it
  volatile int* stop_word = reinterpret_cast<volatile int*>(misc + 8);    // [TG NG], set by a group's own warps
  volatile float* first_lv = reinterpret_cast<volatile float*>(misc + 12);  // log2 vs_0, set by the K producer
  float4* scale_ring = reinterpret_cast<float4*>(gbase + C::kOffScale);   // (ks, log2 ws, 1/ws) per page of a tile
  float* rows = reinterpret_cast<float*>(gbase + C::kOffRow);             // per tile group: n_r,
  float* const row_bias = rows;                                           //
  float* const row_cap = rows + TG * RP;                                  // the highest it may rise to (+inf: no key seen yet),
  float* const row_delta = rows + 2 * TG * RP;                            // a moving bias's step and
  float* const row_fac = rows + 3 * TG * RP;                              // factor; the output factor in the end
  float* const colmax = rows + 4 * TG * RP;                               // [TG][4][RP]
  uint8_t* const row_state = gbase + C::kOffState;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  // Ahead of the barriers' set-up: the producers' first page ids, and the
  // softmax threads' pieces of the query tile.
  const int ppt = T / a.P;   // pages per tile: 2, 4 or 8
  const int tpc = 32 / ppt;  // tiles per chunk of 32 page slots
  // Page id (-1: zero fill) of this lane's slot of chunk k.
  auto chunk_page = [&](int k) -> int {
    const int slot = (tile0 + k * tpc) * ppt + lane;
    if (k * tpc >= n || slot < geo.lo_min / a.P || slot >= (geo.hi_max + a.P - 1) / a.P) return -1;
    const int pg = __ldg(&a.page_table[static_cast<size_t>(b) * a.max_pages + slot]);
    if (pg < 0 || pg >= a.num_pages) {
      flag_status(a.status, DFLASH_STATUS_BAD_PAGE);
      return -1;
    }
    return pg;
  };
  constexpr int CPR = D / 8;  // 8-column pieces of a query row
  constexpr int kPieces = (RP * CPR + kSoft - 1) / kSoft;
  uint4 piece[kPieces];
  const int g_inv = 65536 / a.G + 1;  // r / G = r g_inv >> 16 for r, G <= 128: too large by less than 1 / 128
  int pg_first = -1;
  if (warp < C::kSoftWarps) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int idx = threadIdx.x + i * kSoft;
      const int r = idx / CPR, c = idx % CPR;
      piece[i] = make_uint4(0u, 0u, 0u, 0u);
      if (r < a.R) {
        const int t = (r * g_inv) >> 16;
        piece[i] = __ldg(reinterpret_cast<const uint4*>(
                             a.q + ((static_cast<size_t>(b) * a.K + t) * a.Hq + static_cast<size_t>(h) * a.G + (r - t * a.G)) * D) + c);
      }
    }
  } else if (warp < C::kSoftWarps + 2) {
    pg_first = chunk_page(0);
  }
  if (threadIdx.x == C::kThreads - 32) {  // the PV issuer's first lane
    if constexpr (RERUN)
      for (int e = 0; e < C::kNumBars; ++e) mbar_inval(bars + 8u * e);
    for (int st = 0; st < NSK; ++st) {
      mbar_init(k_full(st), 1);
      mbar_init(k_empty(st), 1);
    }
    for (int st = 0; st < NSV; ++st) {
      mbar_init(v_full(st), 1);
      mbar_init(v_empty(st), 1);
    }
    for (int e = 0; e < C::kRing; ++e) mbar_init(scales_full(e), 1);
    for (int p = 0; p < NB; ++p) {
      mbar_init(s_full(p), 1);
      mbar_init(s_free(p), 4 * NG);
      mbar_init(p_full(p), 4 * NG);
      mbar_init(pv_done(p), 1);
    }
    mbar_init(q_full, C::kSoftWarps);
    *abort_flag = 0;
    *issued_k = 0;
    *issued_v = 0;
    for (int g = 0; g < TG * NG; ++g) stop_word[g] = 0;
    *q_amax = 0;
    *q_rest = 0;
    fence_mbar_init();
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
  }
  if (warp == C::kSoftWarps + 2 && !RERUN) {
    tmem_alloc(smem_u32(misc), C::kTmem);
    tmem_relinquish();
  }
  for (int r = threadIdx.x; r < TG * RP; r += C::kThreads) {
    row_bias[r] = 0.f;
    row_cap[r] = -p8_ninf();
    if (r < RP && !RERUN) row_state[r] = kRowTaken;
  }
  tc_fence_before();
  __syncthreads();  // barriers, row state and the TMEM address are visible
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_launch_dependents();

  if (warp == C::kSoftWarps || warp == C::kSoftWarps + 1) {
    // ------------------------------------------------------------ producers (whole warps)
    const bool is_v = warp != C::kSoftWarps;
    int pg_cur = pg_first, pg_nxt = -1;
    // This lane's page scales, and those of the next chunk (asked for in the
    // chunk's second tile, when their page ids have come).
    float ks_nxt = 1.f, vs_nxt = 1.f;
    auto ask_scales = [&](int pg) {
      ks_nxt = 1.f;
      vs_nxt = 1.f;
      if (pg >= 0) {
        ks_nxt = __ldg(&k_scales[static_cast<size_t>(pg) * a.Hkv + h]);
        vs_nxt = __ldg(&v_scales[static_cast<size_t>(pg) * a.Hkv + h]);
      }
    };
    if (!is_v) ask_scales(pg_cur);
    float4 sc_cur;
    float lv0 = 0.f;  // log2 vs_0
    const uint64_t kv_policy = l2_policy_evict_first();
    const CUtensorMap* map = is_v ? &tm_v : &tm_k;
    const int ns = is_v ? NSV : NSK;
    const uint32_t ring = base + (is_v ? C::kOffV : C::kOffK);
    const uint32_t full0 = is_v ? v_full(0) : k_full(0), empty0 = is_v ? v_empty(0) : k_empty(0);
    volatile int* issued = is_v ? issued_v : issued_k;
    const uint32_t page_bytes = a.P * D;
    const int n_issue = a.withhold_loads ? 0 : n;  // tests of the failure path
    int cur = 0, st = 0, lap = 0, entry = 0, lane0 = 0;
    for (int j = 0; j < n_issue; ++j) {
      if (lane0 == 32) {
        ++cur;
        lane0 = 0;
        pg_cur = pg_nxt;
      }
      if (lap > 0 && !wait_warp(empty0 + 8u * st, (lap - 1) & 1)) {
        if (lane == 0) flag_status(a.status, DFLASH_STATUS_TIMEOUT);
        *abort_flag = 1;
        break;
      }
      if (lane == 0) {
        mbar_arrive_expect_tx(full0 + 8u * st, C::kTile);
        *issued = j + 1;
      }
      __syncwarp();
      const unsigned mine = static_cast<unsigned>(lane - lane0);  // this lane's page of the tile
      if (mine < static_cast<unsigned>(ppt))
        tma_load_4d_hint(ring + st * C::kTile + mine * page_bytes, map, 0, 0, h, pg_cur, full0 + 8u * st, kv_policy);
      if (lane0 == 0) pg_nxt = chunk_page(cur + 1);
      if (!is_v) {
        // The tile's scales.  Entry j % kRing was read for tile j - kRing
        // before its scores were, and QK^T of tile j - NSK, which has
        // completed, waited for the scores of tile j - NSK - NB to be read.
        if (lane0 == 0) {
          const float lv = log2f(vs_nxt);
          if (j == 0) {  // the first page that holds a visible key
            const unsigned have = __ballot_sync(0xffffffffu, pg_cur >= 0);
            lv0 = have != 0 ? __shfl_sync(0xffffffffu, lv, __ffs(have) - 1) : 0.f;
            if (lane == 0) *first_lv = lv0;
          }
          float rel = pg_cur >= 0 ? lv - lv0 : 0.f;
          if (rel < kP8Quietest) rel = kP8Quietest;
          sc_cur = make_float4(ks_nxt, rel, exp2f(-rel), 0.f);
        } else if (lane0 == ppt) {
          ask_scales(pg_nxt);
        }
        if (mine < static_cast<unsigned>(ppt)) scale_ring[entry * 8 + mine] = sc_cur;
        __syncwarp();
        if (lane == 0) mbar_arrive(scales_full(entry));
        if (++entry == C::kRing) entry = 0;
      }
      lane0 += ppt;
      if (++st == ns) {
        st = 0;
        ++lap;
      }
    }
  } else if (warp == C::kSoftWarps + 2) {
    // ------------------------------------------------------------ QK^T issuer
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_e4m3_f32(T, RP, false, false);
      const uint64_t dq = smem_desc_rows(base + C::kOffQ, D, 16, 8 * D);
      const uint64_t dk = smem_desc_rows(base + C::kOffK, D, 16, 8 * D);
      bool ok = mbar_wait(q_full, 0);
      int last = -1, st = 0, lap = 0, buf = 0, blap = 0;
      for (int j = 0; ok && j < n && !*abort_flag; ++j) {
        if (!mbar_wait(k_full(st), lap & 1) || (blap > 0 && !mbar_wait(s_free(buf), (blap - 1) & 1))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t k_off = st * C::kTile;
#pragma unroll
        for (int term = 0; term < 2; ++term)
#pragma unroll
          for (int kk = 0; kk < D / 32; ++kk)
            umma_e4m3(tmem + buf * RP, dk + ((k_off + kk * 32) >> 4), dq + ((term * C::kQ + kk * 32) >> 4), idesc,
                      term + kk > 0 ? 1u : 0u);
        umma_commit(k_empty(st));
        umma_commit(s_full(buf));
        last = j;
        if (++st == NSK) {
          st = 0;
          ++lap;
        }
        if (++buf == NB) {
          buf = 0;
          ++blap;
        }
      }
      if (!ok) {
        flag_status(a.status, DFLASH_STATUS_TIMEOUT);
        *abort_flag = 1;
      }
      // This thread's MMAs have completed before the CTA winds down.
      if (last >= 0) (void)mbar_wait(s_full(last % NB), (last / NB) & 1);
    }
  } else if (warp == C::kSoftWarps + 3) {
    // ------------------------------------------------------------ PV issuer
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_e4m3_f32(D, C::kPCols, true, true);
      const uint64_t dv = smem_desc_rows(base + C::kOffV, D, 16, 8 * D);
      const uint64_t dp = smem_desc_rows(base + C::kOffP, C::kPRow, C::kPBlock, 8 * C::kPRow);
      bool ok = true;
      int last = -1, st = 0, lap = 0, buf = 0, blap = 0, acc = 0;
      for (int j = 0; j < n && !*abort_flag; ++j) {
        if (!mbar_wait(p_full(buf), blap & 1) || !mbar_wait(v_full(st), lap & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t v_off = st * C::kTile;
#pragma unroll
        for (int kk = 0; kk < T / 32; ++kk)
          umma_e4m3(tmem + C::kColO + acc * C::kPCols, dv + ((v_off + kk * 32 * D) >> 4),
                    dp + ((buf * C::kP + kk * 32 * C::kPRow) >> 4), idesc, j >= TG || kk > 0 ? 1u : 0u);
        umma_commit(v_empty(st));
        umma_commit(pv_done(buf));
        last = j;
        if (++st == NSV) {
          st = 0;
          ++lap;
        }
        if (++buf == NB) {
          buf = 0;
          ++blap;
        }
        if (++acc == TG) acc = 0;
      }
      if (!ok) {
        flag_status(a.status, DFLASH_STATUS_TIMEOUT);
        *abort_flag = 1;
      }
      if (last >= 0) (void)mbar_wait(pv_done(last % NB), (last / NB) & 1);
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int tg = warp / (4 * NG);
    const int grp = (warp >> 2) % NG;
    const int quad = warp & 3;
    const int gthread = quad * 32 + lane;  // key of the tile, and thread of the group
    const int bar_id = 1 + (warp >> 2);    // the group's barrier; 15 joins all softmax warps
    const int row0 = grp * NR;             // the group's first row
    float* const my_bias = row_bias + tg * RP + row0;
    float* const my_cap = row_cap + tg * RP + row0;
    float* const my_delta = row_delta + tg * RP + row0;
    float* const my_fac = row_fac + tg * RP + row0;
    float* const my_colmax = colmax + tg * 4 * RP + row0;

    // The query tile: its largest magnitude sets the power of two, then the
    // pieces become codes.
    float inv_qs;
    {
      // Largest finite |q| of a piece, and of its row (pieces in neighbouring
      // lanes), as bits.
      auto piece_top = [&](int i) -> uint32_t {
        const uint32_t w[4] = {piece[i].x, piece[i].y, piece[i].z, piece[i].w};
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t lo = w[e] & 0x7fffu, hi = (w[e] >> 16) & 0x7fffu;
          top = max(top, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
        }
        return top;
      };
      auto row_top = [&](int i) -> uint32_t {
        uint32_t top = piece_top(i);
#pragma unroll
        for (int m = CPR / 2; m >= 1; m >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, m));
        return top;
      };
      if constexpr (RERUN) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          const int r = (threadIdx.x + i * kSoft) / CPR;
          if (r < RP && row_state[r] == kRowDone) piece[i] = make_uint4(0u, 0u, 0u, 0u);
        }
      }
      uint32_t mx = 0, least = 0xffffu;  // least: of the pieces that are not zero
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const uint32_t top = piece_top(i);
        mx = max(mx, top);
        least = min(least, top - 1u);
      }
      mx = __reduce_max_sync(0xffffffffu, mx);
      if (lane == 0) atomicMax(q_amax, mx);
      named_barrier(15, kSoft);
      const uint32_t most = *reinterpret_cast<volatile uint32_t*>(q_amax) >> 7;
      const int eq = min(261 - static_cast<int>(most), 253);
      const float qs = __int_as_float(eq << 23);
      inv_qs = __int_as_float((254 - eq) << 23);
      // Rows far below: seldom a piece, more seldom its row.
      if (__any_sync(0xffffffffu, ((least + 1) >> 7) + kP8Apart < most)) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          const uint32_t top = row_top(i);
          if (top != 0 && (top >> 7) + kP8Apart < most) {
            row_state[(threadIdx.x + i * kSoft) / CPR] = kRowPutOff;
            *q_rest = 1;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int idx = threadIdx.x + i * kSoft;
        const int r = idx / CPR, c = idx % CPR;
        const uint32_t w[4] = {piece[i].x, piece[i].y, piece[i].z, piece[i].w};
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          split_q2(bf16_bits_to_f32(w[e] & 0xffffu) * qs, bf16_bits_to_f32(w[e] >> 16) * qs, hi[e], lo[e]);
        if (r >= RP) break;
        uint8_t* dst = gbase + C::kOffQ + code_word<D>(r, c >> 1) + (c & 1) * 8;
        *reinterpret_cast<uint2*>(dst) = make_uint2(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16));
        *reinterpret_cast<uint2*>(dst + C::kQ) = make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
    }

    const int L = geo.L;
    const float qk_mul = a.scale_log2 * inv_qs;
    // Rows see every key at positions [lo_all, hi_all); a tile reaching
    // outside is masked, by the row interval its key is seen by.
    const int lo_all = a.W > 0 ? max(0, L + a.K - a.W) : 0;
    const int hi_all = L + min(a.K, 1 + a.rw);
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t o_addr = lane_addr + C::kColO + tg * C::kPCols + (C::kOwnBlock ? grp * 128 : 2 * row0);  // O^T: per 8 rows 8 hi columns, then 8 lo
    const int page_of_key = gthread / a.P;
    // P pieces of this key: its 16-byte piece i (rows 8 i .. 8 i + 7 of the
    // group: hi, lo) lies at p_first ^ 16 i of a buffer, with the swizzle of
    // the row length.
    const int p_first = C::kOwnBlock ? grp * C::kPBlock + gthread * 128 + ((gthread & 7) << 4)
                        : C::kPRow == 64 ? gthread * 64 + (((row0 >> 3) ^ ((gthread >> 1) & 3)) << 4)
                                         : gthread * 128 + ((gthread & 7) << 4);
    static_assert(C::kOwnBlock || NG == 1 || RP == 32, "piece addresses");

    float l[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) l[r] = 0.f;

    bool dropped = false;  // a bias fell far with the last tile
    bool bad = false;      // a wait of this warp ran out
    auto failed = [&]() {
      bad = true;
      stop_word[warp >> 2] = 1;
      *abort_flag = 1;
    };
    int entry = tg, elap = 0;
    int k = 0;  // the group's tiles so far
    for (int j = tg; j < n; j += TG, ++k) {
      const int buf = tg + TG * (k & 1);
      const int blap = k >> 1;  // the buffer's uses before this one
      const int p0 = (tile0 + j) * T;
      const int pos = p0 + gthread;
      // The tile's scores and scales.  The P buffer is free once the PV of its
      // last use, two tiles of the group ago, has completed: asked for here,
      // and waited for before the vote if need be.
      const bool got_p = mbar_try_wait(pv_done(buf), (blap - 1) & 1);
      const bool got_s = mbar_try_wait(scales_full(entry), elap & 1) & mbar_try_wait(s_full(buf), blap & 1);
      if (!__all_sync(0xffffffffu, got_s) && !(wait_warp(scales_full(entry), elap & 1) && wait_warp(s_full(buf), blap & 1)))
        failed();
      tc_fence_after();
      uint32_t x[NR];
      load_scores<NR>(lane_addr + buf * RP + row0, x);
      // y = t + n.  The page's log2 ws joins each row's bias in registers: put
      // together in shared memory, one lane a row, it took 1 to 4 % longer (64/4
      // window 99.1 against 95.2 us, 64/16 ragged 607 against 599, of an earlier
      // form).
      const float4 sc = scale_ring[entry * 8 + page_of_key];
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(s_free(buf));
      entry += TG;
      if (entry >= C::kRing) {
        entry -= C::kRing;
        ++elap;
      }
      const float ck = sc.x * qk_mul;
      const float iv = sc.z;
      float y[NR];
#pragma unroll
      for (int q = 0; q < NR / 4; ++q) {
        float4 bb = reinterpret_cast<const float4*>(my_bias)[q];
        add2(bb.x, bb.y, sc.y);
        add2(bb.z, bb.w, sc.y);
        fma2(y[4 * q], y[4 * q + 1], __uint_as_float(x[4 * q]), __uint_as_float(x[4 * q + 1]), ck, bb.x, bb.y);
        fma2(y[4 * q + 2], y[4 * q + 3], __uint_as_float(x[4 * q + 2]), __uint_as_float(x[4 * q + 3]), ck, bb.z, bb.w);
      }
      if (p0 < lo_all || p0 + T > hi_all) {
        asm volatile("" ::: "memory");  // a branch, not selects in every tile
        // Rows [ra, ra + len) see this key: those whose last key is not
        // before it, and whose window reaches it.
        int ra = max(0, pos - L - a.rw) * a.G, rb = a.K * a.G;
        // (Compared first: the sum of a large window and the key's place passes 32 bits.)
        if (a.W > 0 && pos - L < a.K - a.W) rb = (pos - L + a.W) * a.G;
        if (pos >= L + a.K) rb = 0;
        const int len = max(rb - ra, 0);
        ra -= row0;
#pragma unroll
        for (int r = 0; r < NR; ++r)
          if (static_cast<unsigned>(r - ra) >= static_cast<unsigned>(len)) y[r] = p8_ninf();
      }
      float mx = p8_ninf(), mx1 = p8_ninf();
#pragma unroll
      for (int r = 0; r < NR; r += 4) {
        mx = max3(mx, y[r], y[r + 1]);
        mx1 = max3(mx1, y[r + 2], y[r + 3]);
      }
      if (!__all_sync(0xffffffffu, got_p) && !wait_warp(pv_done(buf), (blap - 1) & 1)) failed();
      // Value rows outside the keys the block sees may hold anything: zero
      // them before the PV reads them (boundary tiles only).
      if (grp == 0 && (p0 < geo.lo_min || p0 + T > geo.hi_max)) {
        if (!wait_warp(v_full(j % NSV), (j / NSV) & 1)) {
          failed();
        } else if (pos < geo.lo_min || pos >= geo.hi_max) {
          uint8_t* vrow = gbase + C::kOffV + (j % NSV) * C::kTile + gthread * D;
#pragma unroll
          for (int c = 0; c < D / 16; ++c) *reinterpret_cast<uint4*>(vrow + 16 * c) = make_uint4(0u, 0u, 0u, 0u);
        }
      }
      // The group's first tile sets the biases, its second those of rows whose
      // window starts behind the first.
      const bool look = k <= 1 || dropped || (k % kP8Every == 0 && n - j > kP8Every / 2);
      dropped = false;
      if (barrier_any(bar_id, 128, fmaxf(mx, mx1) > kP8Limit || look || bad)) {
        if (stop_word[warp >> 2] != 0) break;
        // ---- new biases.  Column maxima over the tile's keys, per warp.
#pragma unroll
        for (int r = 0; r < NR; r += 4) {
          const float4 m = make_float4(redux_max(y[r]), redux_max(y[r + 1]), redux_max(y[r + 2]), redux_max(y[r + 3]));
          if (lane == 0) *reinterpret_cast<float4*>(my_colmax + quad * RP + r) = m;
        }
        named_barrier(bar_id, 128);
        float delta = 0.f;
        if (gthread < NR) {
          const int r = gthread;
          const float m0 = my_colmax[r], m1 = my_colmax[RP + r], m2 = my_colmax[2 * RP + r], m3 = my_colmax[3 * RP + r];
          const float a01 = fmaxf(m0, m1), a23 = fmaxf(m2, m3);
          // M = the tile's largest t + n; -inf when the row sees no key of it.
          const float M = fmaxf(a01, a23);
          const float second = fmaxf(fminf(a01, a23), fmaxf(fminf(m0, m1), fminf(m2, m3)));  // the largest of the other warps
          const float old = my_bias[r], cap = my_cap[r];
          const bool first = cap == -p8_ninf();  // O and l of the row are zero so far
          if (M > p8_ninf() && (first || M > kP8Off || (look && M < kP8Low))) {
            const bool alone = M - second > kP8Alone && (first || M > kP8Limit + kP8Alone);
            const float now = fminf(old + ((alone ? kP8Limit : kP8Set) - M), cap);
            delta = now - old;
            my_bias[r] = now;
            my_cap[r] = fminf(cap, now + kP8Rise);
          }
          my_delta[r] = delta;
          my_fac[r] = first ? 1.f : fast_exp2(delta);
        }
        if (barrier_any(bar_id, 128, delta != 0.f)) {
#pragma unroll
          for (int q = 0; q < NR / 4; ++q) {
            const float4 dl = reinterpret_cast<const float4*>(my_delta)[q];
            const float4 fc = reinterpret_cast<const float4*>(my_fac)[q];
            y[4 * q] += dl.x;
            y[4 * q + 1] += dl.y;
            y[4 * q + 2] += dl.z;
            y[4 * q + 3] += dl.w;
            l[4 * q] *= fc.x;
            l[4 * q + 1] *= fc.y;
            l[4 * q + 2] *= fc.z;
            l[4 * q + 3] *= fc.w;
            dropped = dropped || fminf(fminf(dl.x, dl.y), fminf(dl.z, dl.w)) < kP8Drop;
          }
          if (k > 0) {
            // O holds the group's earlier tiles once their PV has completed.
            if (!wait_warp(pv_done(tg + TG * ((k - 1) & 1)), ((k - 1) >> 1) & 1)) failed();
            tc_fence_after();
#pragma unroll 1
            for (int e8 = 0; e8 < NR; e8 += 8) {
              const float4 f0 = *reinterpret_cast<const float4*>(my_fac + e8), f1 = *reinterpret_cast<const float4*>(my_fac + e8 + 4);
              const float f[8] = {f0.x, f0.y, f0.z, f0.w, f1.x, f1.y, f1.z, f1.w};
              bool rest = true;
#pragma unroll
              for (int e = 0; e < 8; ++e) rest = rest && f[e] == 1.f;
              if (rest) continue;  // alike for every thread of the group
              uint32_t o0[8], o1[8];
              tmem_ld8x2_wait(o_addr + 2 * e8, o_addr + 2 * e8 + 8, o0, o1);
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                o0[e] = __float_as_uint(__uint_as_float(o0[e]) * f[e]);
                o1[e] = __float_as_uint(__uint_as_float(o1[e]) * f[e]);
              }
              tmem_st8(o_addr + 2 * e8, o0);
              tmem_st8(o_addr + 2 * e8 + 8, o1);
            }
            tmem_wait_st();
            tc_fence_before();
          }
        }
      }
      uint8_t* pbuf = gbase + C::kOffP + buf * C::kP;
#pragma unroll
      for (int c = 0; c < NR / 8; ++c) {
        uint32_t hi[2], lo[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int r = 8 * c + 4 * q;
          float p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) p[e] = fast_exp2(y[r + e]);
          fma2(l[r], l[r + 1], p[0], p[1], iv, l[r], l[r + 1]);
          fma2(l[r + 2], l[r + 3], p[2], p[3], iv, l[r + 2], l[r + 3]);
          split_p4(p[0], p[1], p[2], p[3], hi[q], lo[q]);
        }
        *reinterpret_cast<uint4*>(pbuf + (p_first ^ (c << 4))) = make_uint4(hi[0], hi[1], lo[0], lo[1]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full(buf));
    }

    // ---- the unit's result, once the group's last PV has completed.
    if (k > 0) {
      if (!wait_warp(pv_done(tg + TG * ((k - 1) & 1)), ((k - 1) >> 1) & 1)) failed();
    }
    if (bad && lane == 0) flag_status(a.status, DFLASH_STATUS_TIMEOUT);
    if (!barrier_any(15, kSoft, bad || stop_word[warp >> 2] != 0)) {
      tc_fence_after();
      // Row sums over the group's keys: lanes, then the four warps.
#pragma unroll
      for (int c = 0; c < NR / 8; ++c) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = l[8 * c + e];
        const float sum = sum8(v, lane);
        if ((lane & 3) == 0) my_colmax[quad * RP + 8 * c + (lane >> 2)] = sum;
      }
      named_barrier(15, kSoft);
      const size_t unit = (static_cast<size_t>(b) * a.Hkv + h) * a.S + s;
      const bool direct = a.S == 1;
      if (threadIdx.x < RP) {
        // One bias for all tile groups: the least (the largest scores).
        const int r = threadIdx.x;
        float sums[TG], least = -p8_ninf();
#pragma unroll
        for (int g = 0; g < TG; ++g) {
          const float* cm = colmax + g * 4 * RP + r;
          sums[g] = (cm[0] + cm[RP]) + (cm[2 * RP] + cm[3 * RP]);
          if (sums[g] != 0.f) least = fminf(least, row_bias[g * RP + r]);
        }
        float sum = 0.f;
#pragma unroll
        for (int g = 0; g < TG; ++g) {
          const float f = sums[g] != 0.f ? fast_exp2(least - row_bias[g * RP + r]) : 0.f;
          row_fac[g * RP + r] = f;
          sum = sums[g] != 0.f ? fmaf(f, sums[g], sum) : sum;
        }
#pragma unroll
        for (int g = 0; g < TG; ++g) row_fac[g * RP + r] *= sum != 0.f ? exp2f(*first_lv) / sum : 0.f;
        const bool taken = r < a.R && row_state[r] == kRowTaken;
        if (!taken) row_delta[r] = __int_as_float(-1);
        if (taken) {
          const float lse = sum > 0.f ? log2f(sum) - least : p8_ninf();
          // Where the row lies in the output, from the first of the block's rows
          // (-1: no row, or one of another pass).
          const int i = (r * g_inv) >> 16, place = i * a.Hq + r - i * a.G;
          row_delta[r] = __int_as_float(place);
          // A row that met a NaN: its partial outputs are NaN, and this
          // weight makes the combine keep them (the LSE becomes -inf).
          if (direct) a.lse2[static_cast<size_t>(b) * a.K * a.Hq + static_cast<size_t>(h) * a.G + place] = lse;
          else a.part_lse[unit * a.R + r] = sum != sum ? -p8_ninf() : lse;
        }
      }
      named_barrier(15, kSoft);
      // O^T: TMEM lane = output column (M = 64 uses 16 lanes of each 32).
      // The groups share the rows, eight at a time.  (Each row's place comes
      // from the table above: with a division by G here, eight an iteration, the
      // output of 128 rows took 17000 cycles.)
      const int d = D == 128 ? gthread : quad * 16 + lane;
      uint16_t* const out = a.out + (static_cast<size_t>(b) * a.K * a.Hq + static_cast<size_t>(h) * a.G) * D;
#pragma unroll 1
      for (int e0 = 8 * (warp >> 2); e0 < a.R; e0 += 8 * TG * NG) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0.f;
#pragma unroll
        for (int g = 0; g < TG; ++g) {
          if (g >= n) break;  // a group without a tile
          uint32_t o0[8], o1[8];
          const uint32_t col = lane_addr + C::kColO + g * C::kPCols + (C::kOwnBlock && e0 >= NR ? 128 + 2 * (e0 - NR) : 2 * e0);
          tmem_ld8x2_wait(col, col + 8, o0, o1);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            v[e] = fmaf(fmaf(__uint_as_float(o1[e]), 1.f / 32.f, __uint_as_float(o0[e])), row_fac[g * RP + e0 + e], v[e]);
        }
        if (D == 128 || lane < 16) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int r = e0 + e, place = __float_as_int(row_delta[r]);
            if (place >= 0) {
              if (direct)
                out[static_cast<size_t>(place) * D + d] = static_cast<uint16_t>(pack_bf16x2(v[e], 0.f) & 0xffffu);
              else
                a.part_o[(unit * a.R + r) * D + d] = v[e];
            }
          }
        }
      }
      tc_fence_before();
    }
  }

  __syncthreads();
  if (*abort_flag && threadIdx.x == 0) {
    const int ik = *issued_k, iv = *issued_v;
    for (int j = ik > NSK ? ik - NSK : 0; j < ik; ++j) (void)mbar_wait(k_full(j % NSK), (j / NSK) & 1);
    for (int j = iv > NSV ? iv - NSV : 0; j < iv; ++j) (void)mbar_wait(v_full(j % NSV), (j / NSV) & 1);
  }
  if (*q_rest && !*abort_flag) {
    // Rows far below the loudest: the unit again, for them alone, once nothing
    // is left in flight on a barrier.
    bool ok = true;
    if (threadIdx.x == 0) {
      for (int j = max(0, n - NSK); ok && j < n; ++j) ok = mbar_wait(k_empty(j % NSK), (j / NSK) & 1);
      for (int j = max(0, n - NSV); ok && j < n; ++j) ok = mbar_wait(v_empty(j % NSV), (j / NSV) & 1);
      for (int j = max(0, n - NB); ok && j < n; ++j)
        ok = mbar_wait(s_full(j % NB), (j / NB) & 1) && mbar_wait(pv_done(j % NB), (j / NB) & 1);
      if (!ok) flag_status(a.status, DFLASH_STATUS_TIMEOUT);
    }
    if (threadIdx.x < RP) {
      const uint8_t st = row_state[threadIdx.x];
      row_state[threadIdx.x] = st == kRowPutOff ? kRowTaken : kRowDone;
    }
    if (__syncthreads_and(ok)) return true;
  }
  __syncthreads();
  if (warp == C::kSoftWarps + 2) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmem);
  }
  return false;
}

// The further passes.  As a function of its own: as a loop around the first pass
// it costs that pass its registers (64/4 window 138 us).
template <int D, int RP>
__device__ __noinline__ void later_passes(const AttnArgs& a, const float* k_scales, const float* v_scales,
                                          const CUtensorMap& tm_k, const CUtensorMap& tm_v) {
  while (unit_pass<D, RP, true>(a, k_scales, v_scales, tm_k, tm_v)) {
  }
}

template <int D, int RP>
__global__ void __launch_bounds__(P8Cfg<D, RP>::kThreads, P8Cfg<D, RP>::kCtas)
    split_page8_kernel(const __grid_constant__ AttnArgs a, const float* __restrict__ k_scales,
                       const float* __restrict__ v_scales, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v) {
  if (unit_pass<D, RP, false>(a, k_scales, v_scales, tm_k, tm_v)) later_passes<D, RP>(a, k_scales, v_scales, tm_k, tm_v);
}

template <int D, int RP>
int launch_t(const AttnArgs& a, const KernelPlan& plan, const float* k_scales, const float* v_scales,
             const CUtensorMap& tm_k, const CUtensorMap& tm_v, cudaStream_t stream) {
  auto kern = split_page8_kernel<D, RP>;
  cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, P8Cfg<D, RP>::kSmem);
  if (err != cudaSuccess) return err;
  return launch_kernel(kern, dim3(plan.S, a.Hkv, a.B), dim3(P8Cfg<D, RP>::kThreads), P8Cfg<D, RP>::kSmem, stream,
                       plan.pdl, a, k_scales, v_scales, tm_k, tm_v);
}

template <int D, int RP>
Page8Shape shape_t() {
  using C = P8Cfg<D, RP>;
  return Page8Shape{RP, C::kThreads, C::kSmem, C::kCtas};
}

// The instantiated row counts: the next one up takes a shape's rows.
#define DFLASH_PAGE8_ROWS(F) F(16) F(32) F(48) F(64) F(96) F(112) F(128)

}  // namespace

int split_page8_tile_keys() { return kP8T; }

Page8Shape split_page8_shape(int D, int R) {
#define CASE(N) \
  if (R <= N) return D == 64 ? shape_t<64, N>() : shape_t<128, N>();
  DFLASH_PAGE8_ROWS(CASE)
#undef CASE
  return Page8Shape{};
}

int launch_split_page8(const AttnArgs& a, const KernelPlan& plan, const float* k_scales, const float* v_scales,
                       const CUtensorMap& tm_k, const CUtensorMap& tm_v, cudaStream_t stream) {
#define CASE(N)                                                                                    \
  if (plan.R_pad == N)                                                                             \
    return a.D == 64 ? launch_t<64, N>(a, plan, k_scales, v_scales, tm_k, tm_v, stream)            \
                     : launch_t<128, N>(a, plan, k_scales, v_scales, tm_k, tm_v, stream);
  DFLASH_PAGE8_ROWS(CASE)
#undef CASE
  return cudaErrorInvalidValue;
}

}  // namespace dflash
