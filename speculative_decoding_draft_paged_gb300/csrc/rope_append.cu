// Rotating append: the new tokens' queries and keys turned by the rotary
// position embedding, and the keys and values written into their page slots,
// in one launch (large calls to E4M3 pages: two that overlap) -- into bf16
// pages, or into E4M3 pages with one scale for each (page, kv head).
//
// Token t of request b (packed rows, j = t - cu[b]) stands at position
// pos = L_b + j, in page slot pos / P at offset pos % P.  With r = rotary_dim
// and the pairs (x1, x2) = (x_i, x_{i + r/2}) or (x_2i, x_2i+1):
//   y1 = x1 c - x2 s,  y2 = x1 s + x2 c,  c = cos_sin[pos][i], s = cos_sin[pos][r/2 + i].
// bf16 outputs are rounded once, from fp32.
//
// E4M3 pages.  The new rows of a page slot (one head of one request) are a
// unit: a = max |y| over them, need = the smallest 2^e (e >= -100) with
// a <= 448 2^e, s = need where the unit starts the page, else max(need, s_old);
// the codes are the nearest E4M3 values of y / s, and where s > s_old the
// kept rows' codes become the nearest of code s_old / s.  Powers of two make
// that second rounding exact but for codes that become subnormal, so a page
// filled token by token keeps its precision.  The nearest value is that of
// the real-number y: fp32 decides it unless y / s lies within fp32's error of
// the border between two codes (one element in 10^5), and then the exact sum
// of the two products is compared with the border in 64 bits.
//
// Bound by bytes (rows in, rows or codes out) where the call is large, by the
// chain lengths -> page table, rows -> maximum -> codes where it is small.  Row
// blocks (queries, and the keys and values of bf16 pages): a few tokens each;
// their positions and page slots are looked up once into shared memory, then a
// thread moves 16 elements of a head (two 16-byte pieces that hold eight
// pairs).  Unit blocks: the rows of a page slot for a few (K or V, head) in
// turn, each held in registers between its maximum and its codes and read once,
// the next one asked for before the maximum of this one is known.  A page slot
// belongs to the block whose chunk of packed tokens holds its first new row.
//
// Measured, replayed in a CUDA graph (bytes over 6.77 TB/s, the rate of a plain
// copy): to bf16 pages, a prompt of 8191 tokens beside eight short ones, 16/1
// heads of 128 69 us, 89 %; 256 blocks of 7 tokens, 64/16 heads of 64 11.0 us,
// 60 %.  To E4M3 pages, 12 prompts of 1 to 4001 tokens, 64/16 heads of 64 107 us,
// 77 %; 64 blocks of 7 tokens, 64/4 heads of 128 6.4 us, 38 %; 256 single tokens,
// 64/4 heads 5.1 us; one token, 16/1 heads 3.3 us.  A call from Python in a loop
// takes 21 to 25 us where the kernel takes less.

#include <cuda_runtime.h>

#include "device_common.cuh"

namespace dflash {
namespace {

constexpr int kMaxRowTokens = 16;
constexpr int kMinScaleExp = -100;
constexpr int kMixedChunk = 16;
// Threads of all unit blocks per SM from which a block takes several heads in
// turn.  1024 / 1536 / 2048 / 4096: 47.9 / 48.2 / 48.2 / 65.7 us (4 prompts of
// 4000 tokens, 8/8 heads of 128), 29.1 / 30.0 / 34.1 / 34.0 (256 blocks of 16
// tokens, 64/16 of 64), 92.2 / 90.2 / 87.0 / 88.3 (12 prompts of 1500, 64/16 of 64).
constexpr long long kUnitThreads = 1536;
// Query items per SM from which the query rows have a launch of their own, with
// the row kernel's occupancy, that the unit blocks overlap.  Apart / together:
// 3.8 / 3.2 us (one token, 16/1 heads), 6.4 / 5.8 (32 blocks of 7, 64/4: 750 per
// SM), 8.4 / 7.5 (2000 tokens, 16/1: 1700), 12.3 / 12.3 (128 blocks of 7, 64/4:
// 3000), 20.3 / 21.9 (256 of them), 31 / 45 (a prompt of 4000, 64/4).
constexpr long long kRowsApart = 2048;

// Where token t belongs: request b and its rows, or b = -1 (a row behind the
// last sequence, before the first, past the bound on a request's rows, or
// cu_tokens that do not increase).  long_request: rows past the bound exist.
struct TokenPlace {
  int b, first, end;
  bool long_request;
};

// Whole warp, t alike in every lane: 32 probes a round.
__device__ __forceinline__ TokenPlace find_token(const RopeAppendArgs& a, int t) {
  TokenPlace p;
  if (a.cu_tokens == nullptr) {
    const int n = a.T / a.B;
    p.b = t / n;
    p.first = p.b * n;
    p.end = p.first + n;
    p.long_request = false;
    return p;
  }
  const int lane = threadIdx.x & 31;
  int lo = 0, len = a.B;  // the last b in [lo, lo + len) with cu[b] <= t
  while (len > 1) {
    const int step = (len + 31) >> 5;
    const int at = lo + lane * step;
    const bool le = lane * step < len && __ldg(&a.cu_tokens[at]) <= t;
    const unsigned m = __ballot_sync(0xffffffffu, le);
    const int k = m == 0 ? 0 : 31 - __clz(m);
    len = min(step, len - k * step);
    lo += k * step;
  }
  p.b = lo;
  p.first = __ldg(&a.cu_tokens[lo]);
  p.end = min(__ldg(&a.cu_tokens[lo + 1]), a.T);
  p.long_request = p.first >= 0 && p.end > p.first && p.end - p.first > a.max_new;
  if (p.long_request) p.end = p.first + a.max_new;
  if (p.first < 0 || t < p.first || t >= p.end) p.b = -1;
  return p;
}

__device__ __forceinline__ int clamped_len(const RopeAppendArgs& a, int b, bool flag) {
  const int L = __ldg(&a.ctx_lens[b]);
  if (L >= 0 && L <= a.max_ctx_len) return L;
  if (flag && a.status != nullptr) flag_status(a.status, DFLASH_STATUS_BAD_CTX_LEN);
  return L < 0 ? 0 : a.max_ctx_len;
}

// Two 16-byte pieces -> 16 numbers, and eight numbers -> one.
__device__ __forceinline__ void unpack16(const uint4& w0, const uint4& w1, float (&x)[16]) {
  const uint32_t u[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    x[2 * e] = bf16_bits_to_f32(u[e] & 0xffffu);
    x[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}

// Item i of a head row: the two 8-element pieces (their indices) that hold
// eight whole pairs, or two pieces that are not rotated.
struct Item {
  int c0, c1;
  bool turned;
};

__device__ __forceinline__ Item item_of(int i, int rd, bool interleaved) {
  Item it;
  const int hc = rd >> 4;  // pieces per half = items that are rotated
  it.turned = i < hc;
  if (it.turned && !interleaved) {
    it.c0 = i;
    it.c1 = i + hc;
  } else {
    it.c0 = 2 * i;
    it.c1 = 2 * i + 1;
  }
  return it;
}

// cos and sin of an item's eight pairs: entries 8i .. 8i + 7 of each half of
// the position's row in both pair orders.
__device__ __forceinline__ void load_angles(const RopeAppendArgs& a, int pos, int i, float (&c)[8], float (&s)[8]) {
  const float4* row = reinterpret_cast<const float4*>(a.cos_sin + static_cast<size_t>(pos) * a.rotary_dim + 8 * i);
  const float4* row2 = reinterpret_cast<const float4*>(a.cos_sin + static_cast<size_t>(pos) * a.rotary_dim + (a.rotary_dim >> 1) + 8 * i);
  const float4 c0 = __ldg(row), c1 = __ldg(row + 1), s0 = __ldg(row2), s1 = __ldg(row2 + 1);
  c[0] = c0.x; c[1] = c0.y; c[2] = c0.z; c[3] = c0.w; c[4] = c1.x; c[5] = c1.y; c[6] = c1.z; c[7] = c1.w;
  s[0] = s0.x; s[1] = s0.y; s[2] = s0.z; s[3] = s0.w; s[4] = s1.x; s[5] = s1.y; s[6] = s1.z; s[7] = s1.w;
}

// Pair k of an item's elements x[0..7] (first piece), x[8..15] (second).
template <bool INTER>
__device__ __forceinline__ void turn(float (&x)[16], const float (&c)[8], const float (&s)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int p = INTER ? 2 * k : k, q = INTER ? 2 * k + 1 : 8 + k;
    const float x1 = x[p], x2 = x[q];
    x[p] = fmaf(x1, c[k], -(x2 * s[k]));
    x[q] = fmaf(x1, s[k], x2 * c[k]);
  }
}

// ---------------------------------------------------------------- row blocks

// Tokens [t0, t0 + nt): the query rows, and (bf16 pages) the key and value
// rows.  Thread: item i of every (NT / ipr)-th row of the nt tokens; the first
// is asked for before the places are known.  One item at a time and many
// threads: two, three or four at a time need 1.5 to 2 times the registers and
// took 73, 79 and 85 us against 67 (a prompt of 8191 tokens beside eight
// short ones).
template <int NT, bool INTER>
__device__ __forceinline__ void row_block(const RopeAppendArgs& a, int t0, int nt) {
  __shared__ int s_pos[kMaxRowTokens], s_page[kMaxRowTokens];  // pos -1: no row
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ipr = a.D >> 4;  // items per head row: 4 or 8
  const int i = threadIdx.x % ipr;
  const int q_rows = a.q != nullptr ? a.Hq : 0;
  const unsigned rows = q_rows + (a.kv_rows ? 2 * a.Hkv : 0);
  const unsigned total = nt * rows;
  uint4 w0, w1;
  auto load = [&](unsigned vr) {
    const unsigned k = vr / rows;
    const int row = vr - k * rows;
    const size_t t = t0 + k;
    const int kv = row - q_rows;
    const bool is_v = kv >= a.Hkv;
    const uint16_t* src = kv < 0 ? a.q + t * a.q_stride + row * a.D
                                 : (is_v ? a.v + t * a.v_stride + (kv - a.Hkv) * a.D : a.k + t * a.k_stride + kv * a.D);
    const Item it = item_of(i, is_v ? 0 : a.rotary_dim, INTER);
    w0 = *(reinterpret_cast<const uint4*>(src) + it.c0);
    w1 = *(reinterpret_cast<const uint4*>(src) + it.c1);
  };
  unsigned vr = threadIdx.x / ipr;
  if (vr < total) load(vr);
  for (int k = warp; k < nt; k += NT / 32) {
    const int t = t0 + k;
    const TokenPlace p = find_token(a, t);
    if (lane == 0) {
      int pos = -1, page = -1;
      if (p.b >= 0) {
        pos = clamped_len(a, p.b, true) + t - p.first;
        if (p.long_request && a.status != nullptr) flag_status(a.status, DFLASH_STATUS_BAD_TOKENS);
        if (a.rotary_dim > 0 && pos >= a.num_positions) {
          if (a.status != nullptr) flag_status(a.status, DFLASH_STATUS_BAD_TOKENS);
          pos = -1;
        } else if (a.kv_rows) {
          const int slot = pos / a.P;
          page = slot < a.max_pages ? __ldg(&a.page_table[static_cast<size_t>(p.b) * a.max_pages + slot]) : -1;
          if (page < 0 || page >= a.num_pages) {
            if (a.status != nullptr) flag_status(a.status, DFLASH_STATUS_BAD_PAGE);
            page = -1;
          }
        }
      }
      s_pos[k] = pos;
      s_page[k] = page;
    }
  }
  __syncthreads();
  while (vr < total) {
    const unsigned k = vr / rows;
    const int row = vr - k * rows;
    const int pos = s_pos[k];
    const int kv = row - q_rows;
    const bool is_v = kv >= a.Hkv;
    if (pos >= 0 && (kv < 0 || s_page[k] >= 0)) {
      uint16_t* dst;
      if (kv < 0) {
        dst = a.q_out + ((t0 + static_cast<size_t>(k)) * a.Hq + row) * a.D;
      } else {
        const int hh = is_v ? kv - a.Hkv : kv;
        dst = static_cast<uint16_t*>(is_v ? a.v_pages : a.k_pages) +
              ((static_cast<size_t>(s_page[k]) * a.Hkv + hh) * a.P + pos % a.P) * a.D;
      }
      const Item it = item_of(i, is_v ? 0 : a.rotary_dim, INTER);
      if (it.turned) {
        float c[8], s[8], x[16];
        load_angles(a, pos, i, c, s);
        unpack16(w0, w1, x);
        turn<INTER>(x, c, s);
        w0 = pack8(x);
        w1 = pack8(x + 8);
      }
      *(reinterpret_cast<uint4*>(dst) + it.c0) = w0;
      *(reinterpret_cast<uint4*>(dst) + it.c1) = w1;
    }
    vr += NT / ipr;
    if (vr < total) load(vr);
  }
}

// ---------------------------------------------------------------- unit blocks

// Numbers next to the border between two E4M3 values.  u = |v| (plus 2^-6
// below 2^-6, which gives those numbers the one spacing 2^-9) lies between two
// neighbours with three mantissa bits; their middle is the border.
struct Border {
  uint32_t low;  // code of the lower neighbour, without sign
  float mid;     // the middle, in units of the scale
  float dist;    // |u - middle|
};
__device__ __forceinline__ Border border_of(float v) {
  float u = fabsf(v);
  const bool small = u < 0.015625f;
  if (small) u += 0.015625f;
  const float mid = __uint_as_float((__float_as_uint(u) & 0xfff00000u) | 0x00080000u);
  Border r;
  r.low = (__float_as_uint(u) >> 20) - (120u << 3) - (small ? 8u : 0u);
  r.mid = small ? mid - 0.015625f : mid;
  r.dist = fabsf(u - mid);
  return r;
}

// Whether v, off by at most err, could lie on either side of the border (the
// sum with 2^-6 rounds by 2^-30 at most).
__device__ __forceinline__ bool near_border(float v, float err) {
  return border_of(v).dist <= err + (fabsf(v) < 0.015625f ? 1.8626451e-9f : 0.f);
}

// Code of y / s where v = y / s but for fp32's error lies next to a border:
// |y| against border * s, exact in 64 bits (5 and 24 significant bits).
__device__ __forceinline__ uint32_t code_at_border(double y, float s, float v) {
  const Border b = border_of(v);
  const double edge = static_cast<double>(b.mid) * static_cast<double>(s), m = fabs(y);
  const uint32_t code = b.low + ((m > edge || (m == edge && (b.low & 1u))) ? 1u : 0u);
  return min(code, 0x7eu) | (signbit(y) ? 0x80u : 0u);
}

// Element e (0..15) of an item in 64 bits, from its inputs: the products are
// exact there, and their sum is to 2^-53.
__device__ __forceinline__ double element_exact(const RopeAppendArgs& a, const uint16_t* row, const Item& it, int pos, int i,
                                                bool inter, int e) {
  auto x = [&](int k) -> double { return bf16_bits_to_f32(row[8 * (k < 8 ? it.c0 : it.c1) + (k & 7)]); };
  if (!it.turned) return x(e);
  const int k = inter ? e >> 1 : e & 7;
  const bool second = inter ? (e & 1) != 0 : e >= 8;
  const int p = inter ? 2 * k : k, q = inter ? 2 * k + 1 : 8 + k;
  const float* ang = a.cos_sin + static_cast<size_t>(pos) * a.rotary_dim + 8 * i + k;
  const double c = ang[0], sn = ang[a.rotary_dim >> 1];
  return second ? x(p) * sn + x(q) * c : x(p) * c - x(q) * sn;
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

// Exponent e of the smallest power of two with m <= 448 * 2^e (m finite > 0
// in fp32): 448 = 1.75 * 2^8.
__device__ __forceinline__ int scale_exp(float m) {
  const uint32_t bits = __float_as_uint(m) + 0x1fffffu;  // past 1.75 carries into the exponent
  return max(static_cast<int>(bits >> 23) - 127 - 8, kMinScaleExp);
}

// A power of two whose reciprocal is a normal number too.
__device__ __forceinline__ bool is_pow2(float s) {
  return (__float_as_uint(s) & 0x7fffffu) == 0 && s < 8.5070592e37f;  // 2^126
}

// max(m, |a|, |b|), NaN where one of them is.
__device__ __forceinline__ float max_abs3(float m, float a, float b) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(m), "f"(a), "f"(b));
  return d;
}

// The page slots whose first new row lies in chunk `chunk`, for the (K or V,
// head) pairs [j0, j1) of the 2 Hkv, K's first.  ROWS: the most rows of a unit;
// NT: the threads that take one, tid among them (the whole block, or one warp).
template <int D, int ROWS, int NT, bool INTER>
__device__ __forceinline__ void unit_block(const RopeAppendArgs& a, int chunk, int j0, int j1) {
  const int tid = threadIdx.x % NT;
  constexpr int IPR = D / 16;
  constexpr int kItems = ROWS * IPR / NT;  // per thread
  constexpr int kWarps = NT / 32;
  __shared__ uint32_t s_max[2][kWarps];  // bits of a warp's maximum; the sign: a number that is not finite
  __shared__ double s_maxd[kWarps];
  const int warp = tid >> 5, lane = tid & 31;
  const int t_end = min((chunk + 1) * a.chunk_tokens, a.T);
  int t = chunk * a.chunk_tokens;
  int par = 0;  // half of s_max in use
  while (t < t_end) {
    const TokenPlace p = find_token(a, t);
    if (p.b < 0) {
      // A row of no request: behind the last one there are only more of them.
      if (a.cu_tokens == nullptr || t >= __ldg(&a.cu_tokens[a.B])) break;
      ++t;
      continue;
    }
    const bool first = tid == 0 && j0 == 0;
    const int pos = clamped_len(a, p.b, first && t == p.first) + t - p.first;
    if (p.long_request && first && t == p.first && a.status != nullptr) flag_status(a.status, DFLASH_STATUS_BAD_TOKENS);
    const int off = pos % a.P;
    const int n_slot = min(a.P - off, p.end - t);
    const int t0 = t;
    t += n_slot;
    if (off != 0 && t0 != p.first) continue;  // the slot started in an earlier chunk
    const int slot = pos / a.P;
    const int page = slot < a.max_pages ? __ldg(&a.page_table[static_cast<size_t>(p.b) * a.max_pages + slot]) : -1;
    int rows = n_slot;
    if (a.rotary_dim > 0 && pos > a.num_positions - rows) {
      if (first && a.status != nullptr) flag_status(a.status, DFLASH_STATUS_BAD_TOKENS);
      rows = a.num_positions - pos;
      if (rows <= 0) continue;
    }
    // This thread's items of a unit: row rr, item i of it (the same for every head).
    const int n_items = rows * IPR;
    uint4 w0[kItems], w1[kItems];  // the pair about to be taken, as loaded
    auto load = [&](int j) {
      const bool is_v = j >= a.Hkv;
      const int h = is_v ? j - a.Hkv : j;
      const uint16_t* src = is_v ? a.v : a.k;
      const size_t stride = is_v ? a.v_stride : a.k_stride;
#pragma unroll
      for (int m = 0; m < kItems; ++m) {
        const int idx = tid + m * NT;
        if (idx < n_items) {
          const Item it = item_of(idx % IPR, is_v ? 0 : a.rotary_dim, INTER);
          const uint4* row = reinterpret_cast<const uint4*>(src + (t0 + idx / IPR) * stride + h * D);
          w0[m] = __ldg(row + it.c0);
          w1[m] = __ldg(row + it.c1);
        }
      }
    };
    load(j0);
    if (page < 0 || page >= a.num_pages) {
      if (first && a.status != nullptr) flag_status(a.status, DFLASH_STATUS_BAD_PAGE);
      continue;
    }
    const size_t unit0 = static_cast<size_t>(page) * a.Hkv;
    auto stored = [&](int j) -> float {
      return off > 0 ? __ldcg(j >= a.Hkv ? &a.v_scales[unit0 + j - a.Hkv] : &a.k_scales[unit0 + j]) : 0.f;
    };
    float s_next = stored(j0);
#pragma unroll 1
    for (int j = j0; j < j1; ++j) {
      const bool is_v = j >= a.Hkv;
      const int h = is_v ? j - a.Hkv : j;
      const int rd = is_v ? 0 : a.rotary_dim;
      float s_old = s_next;
      float y[kItems][16];
      float mx = 0.f;
#pragma unroll
      for (int m = 0; m < kItems; ++m) {
        const int idx = tid + m * NT;
        if (idx < n_items) {
          const int i = idx % IPR;
          unpack16(w0[m], w1[m], y[m]);
          if (item_of(i, rd, INTER).turned) {
            float c[8], sn[8];
            load_angles(a, pos + idx / IPR, i, c, sn);
            turn<INTER>(y[m], c, sn);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) mx = max_abs3(mx, y[m][2 * e], y[m][2 * e + 1]);
        }
      }
      bool bad = !(mx <= 3.4028235e38f);
      if (bad) {  // the largest of the finite ones
        mx = 0.f;
#pragma unroll
        for (int m = 0; m < kItems; ++m) {
          if (tid + m * NT < n_items) {
#pragma unroll
            for (int e = 0; e < 16; ++e) mx = fmaxf(mx, fabsf(y[m][e]) <= 3.4028235e38f ? fabsf(y[m][e]) : 0.f);
          }
        }
      }
      if (j + 1 < j1) {
        load(j + 1);
        s_next = stored(j + 1);
      }
      // The unit's largest magnitude.
      mx = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mx)));  // non-negative: ordered as integers
      bad = __any_sync(0xffffffffu, bad);
      uint32_t top = __float_as_uint(mx), any_bad = bad ? 1 : 0;
      if constexpr (kWarps > 1) {
        if (lane == 0) s_max[par][warp] = top | (any_bad << 31);
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          top = max(top, s_max[par][w] & 0x7fffffffu);
          any_bad |= s_max[par][w] >> 31;
        }
        par ^= 1;
      }
      mx = __uint_as_float(top);
      const uint16_t* src = is_v ? a.v : a.k;
      const size_t stride = is_v ? a.v_stride : a.k_stride;
      int ex = mx > 0.f ? scale_exp(mx) : kMinScaleExp;
      // A rotated maximum within fp32's error of 448 * 2^e: decided in 64 bits.
      const uint32_t man = (__float_as_uint(mx) & 0x7fffffu) - (0x600000u - 8u);
      if (rd > 0 && man <= 16u && mx > 0.f) {
        double md = 0.0;
#pragma unroll 1
        for (int idx = tid; idx < n_items; idx += NT) {
          const int rr = idx / IPR, i = idx % IPR;
#pragma unroll 1
          for (int e = 0; e < 16; ++e) {
            const double v = fabs(element_exact(a, src + (t0 + rr) * stride + h * D, item_of(i, rd, INTER), pos + rr, i, INTER, e));
            if (v <= 3.4028234663852886e38) md = fmax(md, v);
          }
        }
#pragma unroll
        for (int k = 16; k >= 1; k >>= 1) md = fmax(md, __shfl_xor_sync(0xffffffffu, md, k));
        if constexpr (kWarps > 1) {
          if (lane == 0) s_maxd[warp] = md;
          __syncthreads();
          for (int w = 0; w < kWarps; ++w) md = fmax(md, s_maxd[w]);
          __syncthreads();  // before another unit writes s_maxd
        }
        const int e0 = max(static_cast<int>(__float_as_uint(mx) >> 23) - 127 - 8, kMinScaleExp);
        ex = md <= 448.0 * static_cast<double>(__int_as_float((e0 + 127) << 23)) ? e0 : e0 + 1;
      }
      const float need = __int_as_float((ex + 127) << 23);
      bool bad_scale = false;
      if (off > 0 && !(s_old > 0.f && s_old <= 3.4028235e38f)) {
        s_old = __int_as_float((kMinScaleExp + 127) << 23);  // a stored scale that is no scale
        bad_scale = true;
      }
      const float s = off > 0 ? fmaxf(need, s_old) : need;
      const bool pow2 = is_pow2(s);
      const float inv = pow2 ? __int_as_float((254 << 23) - __float_as_int(s)) : 0.f;
      if (tid == 0) {
        (is_v ? a.v_scales : a.k_scales)[unit0 + h] = s;
        if ((any_bad || bad_scale) && a.status != nullptr) flag_status(a.status, DFLASH_STATUS_FP8_RANGE);
      }
      uint8_t* base = static_cast<uint8_t*>(is_v ? a.v_pages : a.k_pages) + (unit0 + h) * a.P * D;
#pragma unroll
      for (int m = 0; m < kItems; ++m) {
        const int idx = tid + m * NT;
        if (idx < n_items) {
          const int rr = idx / IPR, i = idx % IPR;
          const Item it = item_of(i, rd, INTER);
          float v[16];
          if (pow2) {
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = y[m][e] * inv;
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = y[m][e] / s;
          }
          // fp32 error of an element: half an ulp each of one product, the sum
          // and a division (2^-24 of at most |v1| + |v2|: a product is at most
          // |(x1, x2)| times the larger of |c| and |s|), and half an ulp of
          // the sums below.  Where v - err and v + err, of every element, have
          // one code, it is that of the real number; all else is looked at
          // element by element.
          constexpr float kErr = 2.9802322e-7f;  // 5 * 2^-24
          uint32_t code[4], apart = 1;
          if (it.turned && !any_bad) {
            apart = 0;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              float up[4], down[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int at = 4 * q + e;
                const float err = (fabsf(v[at]) + fabsf(v[INTER ? at ^ 1 : at ^ 8])) * kErr;
                up[e] = v[at] + err;
                down[e] = v[at] - err;
              }
              code[q] = e4m3x4(up[0], up[1], up[2], up[3]);
              apart |= code[q] ^ e4m3x4(down[0], down[1], down[2], down[3]);
            }
          }
          uint32_t close = 0;  // elements next to a border
          if (apart != 0) {
#pragma unroll
            for (int q = 0; q < 4; ++q) code[q] = e4m3x4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
            if (it.turned || !pow2) {
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const float other = it.turned ? fabsf(v[INTER ? e ^ 1 : e ^ 8]) : 0.f;
                close |= near_border(v[e], (fabsf(v[e]) + other) * kErr) ? 1u << e : 0u;
              }
            }
          }
          uint8_t* dst = base + (off + rr) * D;
          *reinterpret_cast<uint2*>(dst + 8 * it.c0) = make_uint2(code[0], code[1]);
          *reinterpret_cast<uint2*>(dst + 8 * it.c1) = make_uint2(code[2], code[3]);
#pragma unroll 1
          while (close != 0) {
            const int e = __ffs(close) - 1;
            close &= close - 1;
            const double ye = element_exact(a, src + (t0 + rr) * stride + h * D, it, pos + rr, i, INTER, e);
            dst[8 * (e < 8 ? it.c0 : it.c1) + (e & 7)] =
                static_cast<uint8_t>(code_at_border(ye, s, static_cast<float>(ye) / s));
          }
        }
      }
      // Kept rows under a scale that grew.
      if (off > 0 && s > s_old) {
        const bool shift = pow2 && is_pow2(s_old);
        const float ratio = s_old * inv;  // exact when both are powers of two
#pragma unroll 4
        for (int idx = tid; idx < off * (D / 16); idx += NT) {
          uint4* at = reinterpret_cast<uint4*>(base) + idx;
          const uint4 c = *at;
          uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint2 f = e4m3x4_to_f16x4(w[e]);
            const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&f.x));
            const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&f.y));
            if (shift) {
              w[e] = e4m3x4(f0.x * ratio, f0.y * ratio, f1.x * ratio, f1.y * ratio);
            } else {
              const float q[4] = {f0.x * s_old / s, f0.y * s_old / s, f1.x * s_old / s, f1.y * s_old / s};
              const float fc[4] = {f0.x, f0.y, f1.x, f1.y};
              w[e] = e4m3x4(q[0], q[1], q[2], q[3]);
              for (int k = 0; k < 4; ++k)
                if (near_border(q[k], fabsf(q[k]) * 2.3841858e-7f))
                  w[e] = (w[e] & ~(0xffu << (8 * k))) |
                         (code_at_border(static_cast<double>(fc[k]) * static_cast<double>(s_old), s, q[k]) << (8 * k));
            }
          }
          *at = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
  }
}

// bf16 pages: row blocks only.
template <bool INTER>
__global__ void __launch_bounds__(256, 6) rope_rows_kernel(const RopeAppendArgs a) {
  pdl_launch_dependents();
  const int t0 = blockIdx.x * a.row_tokens;
  row_block<256, INTER>(a, t0, min(a.row_tokens, a.T - t0));
}

// E4M3 pages: blocks y < unit_blocks of a chunk take unit_heads (K or V, head)
// pairs of it for each of their kThreads / kUnit parts, the others (if any) the
// query rows of row_tokens tokens.
// Forms, by the most rows of a unit (what a thread keeps is what a unit waits
// for, so a unit gets as many threads as it has items where the card has room):
//   kFewRows (4 rows of 128, 8 of 64): a warp takes a unit, no block barrier.
//     Against the 16-row form 5.1 / 9.7 us (256 single tokens, 64/4 heads of
//     128), 6.0 / 7.5 (64 blocks of 4, 64/16 of 64).
//   kRows16: an item a thread.  With the 64-row form 64 blocks of 7 tokens, 64/4
//     heads of 128, took 9.4 us, with this one 7.7.
//   kRows32: the same; kRows32Many: two items a thread, where the units fill
//     the card: half the threads to share a unit's scale.  Many / one item: 81 /
//     90 us (12 prompts of 1500, 64/16 heads of 64), 54.7 / 55.3 (8 of 1000, 64/4
//     of 128), but 7.0 / 6.3 (one of 500, 64/16) below.
//   kRows64: two items a thread.
// Threads per SM, which set the registers: 768 / 896 / 1024 at D = 128 7.0 / 6.5 /
// 6.7 us (64 blocks of 7 tokens, 64/4 heads) and 20.0 / 18.9 / 18.6 (256), but
// 896 at D = 64 98 against 90 (12 prompts of 1500, 64/16).
enum UnitForm { kFewRows, kRows16, kRows32, kRows32Many, kRows64 };
template <int D, UnitForm FORM>
struct UnitCfg {
  static constexpr int kRows = FORM == kFewRows ? 512 / D : (FORM == kRows16 ? 16 : (FORM == kRows64 ? 64 : 32));
  static constexpr int kUnit = FORM == kFewRows ? 32 : (FORM == kRows16 || FORM == kRows32Many ? D : 2 * D);  // threads per unit
  static constexpr int kThreads = FORM == kFewRows ? 128 : kUnit;
  static constexpr int kBlocks = (FORM == kRows64 ? 512 : (FORM == kRows32Many ? 640 : (D == 128 ? 896 : 768))) / kThreads;
};
template <int D, UnitForm FORM, bool INTER>
__global__ void __launch_bounds__(UnitCfg<D, FORM>::kThreads, UnitCfg<D, FORM>::kBlocks) append_units_kernel(const RopeAppendArgs a) {
  using C = UnitCfg<D, FORM>;
  pdl_launch_dependents();
  const int y = blockIdx.y;
  if (y < a.unit_blocks) {
    const int j0 = (y * (C::kThreads / C::kUnit) + static_cast<int>(threadIdx.x) / C::kUnit) * a.unit_heads;
    if (j0 < 2 * a.Hkv) unit_block<D, C::kRows, C::kUnit, INTER>(a, blockIdx.x, j0, min(j0 + a.unit_heads, 2 * a.Hkv));
  } else {
    const int t0 = blockIdx.x * a.chunk_tokens + (y - a.unit_blocks) * a.row_tokens;
    const int nt = min(min(a.row_tokens, (static_cast<int>(blockIdx.x) + 1) * a.chunk_tokens - t0), a.T - t0);
    if (nt > 0) row_block<C::kThreads, INTER>(a, t0, nt);
  }
  // Where the query rows have a launch of their own just before, nothing here
  // depends on it, and these blocks overlap it; but what follows this launch
  // may read the queries.
  pdl_wait_primary();
}

// Tokens of a row block: about four items a thread (one and three: 110 and 69 us
// against 67 for the prompts above; eight: 13.1 against 10.8 us for 256 blocks
// of 7 tokens, 64/16 heads).
int row_block_tokens(int items_per_token, int threads) {
  const int n = 4 * threads / items_per_token;
  return n < 1 ? 1 : (n > kMaxRowTokens ? kMaxRowTokens : n);
}

// Query rows, and (kv_rows) the key and value rows.
cudaError_t launch_rows(RopeAppendArgs a, int kv_rows, cudaStream_t stream) {
  a.kv_rows = kv_rows;
  a.row_tokens = row_block_tokens(a.D / 16 * ((a.q != nullptr ? a.Hq : 0) + (kv_rows ? 2 * a.Hkv : 0)), 256);
  const unsigned grid = static_cast<unsigned>((a.T + a.row_tokens - 1) / a.row_tokens);
  if (a.interleaved) rope_rows_kernel<true><<<grid, 256, 0, stream>>>(a);
  else rope_rows_kernel<false><<<grid, 256, 0, stream>>>(a);
  return cudaGetLastError();
}

template <int D, UnitForm FORM>
cudaError_t launch_units(RopeAppendArgs a, int num_sms, cudaStream_t stream) {
  using C = UnitCfg<D, FORM>;
  const int chunks = (a.T + a.chunk_tokens - 1) / a.chunk_tokens;
  // Pairs that a part takes in turn: one while that leaves the card room, then
  // as many as keep the threads of all blocks at kUnitThreads per SM, alike in
  // every part.
  const long long pairs = static_cast<long long>(chunks) * 2 * a.Hkv;
  const long long most = pairs * C::kUnit / (kUnitThreads * num_sms);
  const int parts = static_cast<int>(most <= 1 ? 2 * a.Hkv : (2 * a.Hkv + most - 1) / most);
  a.unit_heads = (2 * a.Hkv + parts - 1) / parts;
  const int per_block = a.unit_heads * (C::kThreads / C::kUnit);
  a.unit_blocks = (2 * a.Hkv + per_block - 1) / per_block;
  int row_blocks = 0;
  bool apart = false;
  if (a.q != nullptr) {
    apart = static_cast<long long>(a.T) * a.Hq * (D / 16) >= kRowsApart * num_sms || a.unit_blocks > 65535 - 64;
    if (apart) {
      const cudaError_t err = launch_rows(a, 0, stream);
      if (err != cudaSuccess) return err;
    } else {
      a.row_tokens = row_block_tokens(D / 16 * a.Hq, C::kThreads);
      row_blocks = (a.chunk_tokens + a.row_tokens - 1) / a.row_tokens;
    }
  }
  return launch_kernel(a.interleaved ? append_units_kernel<D, FORM, true> : append_units_kernel<D, FORM, false>,
                       dim3(chunks, a.unit_blocks + row_blocks), dim3(C::kThreads), 0, stream, apart, a);
}

template <int D>
cudaError_t launch_units_d(const RopeAppendArgs& a, int rows, int num_sms, cudaStream_t stream) {
  if (rows <= UnitCfg<D, kFewRows>::kRows) return launch_units<D, kFewRows>(a, num_sms, stream);
  if (rows <= 16) return launch_units<D, kRows16>(a, num_sms, stream);
  if (rows > 32) return launch_units<D, kRows64>(a, num_sms, stream);
  const long long pairs = static_cast<long long>((a.T + a.chunk_tokens - 1) / a.chunk_tokens) * 2 * a.Hkv;
  return pairs * 2 * D >= kUnitThreads * num_sms ? launch_units<D, kRows32Many>(a, num_sms, stream)
                                                 : launch_units<D, kRows32>(a, num_sms, stream);
}

}  // namespace

int launch_rope_append(const RopeAppendArgs& a_in, int num_sms, cudaStream_t stream) {
  if (a_in.k_scales == nullptr) return launch_rows(a_in, 1, stream);
  RopeAppendArgs a = a_in;
  a.kv_rows = 0;
  const int rows = a.max_new < a.P ? a.max_new : a.P;  // the most of a unit
  // Tokens of a chunk: those of a unit, but a block takes the units that start
  // in its chunk one after the other, so no more than the mean of the requests,
  // and where more than kMixedChunk requests of different lengths could start in
  // it no more than that.  Chunks of a unit's rows / of the mean / capped, too:
  // 119 / 39.5 / 39.5 us (256 single tokens and a prompt of 2000, 64/4 heads of
  // 128), 58.7 / 58.3 / 37.9 (64 and the same, 64/16 of 64), 31.3 / 31.3 / 28.7
  // (64 of 1 to 200, 8/8 of 128), but 87.2 / 87.4 / 88.1 (12 prompts of 1 to
  // 4000, so not capped; at 8 they take 97).
  const int mean = (a.T + a.B - 1) / a.B;
  a.chunk_tokens = mean < rows ? mean : rows;
  if (a.cu_tokens != nullptr && a.B > kMixedChunk && a.chunk_tokens > kMixedChunk) a.chunk_tokens = kMixedChunk;
  return a.D == 64 ? launch_units_d<64>(a, rows, num_sms, stream) : launch_units_d<128>(a, rows, num_sms, stream);
}

}  // namespace dflash
