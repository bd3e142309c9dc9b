// cache_attention.hip -- attention over the paged 4-bit cache (cache.hpp).
//
// Per query head, with its head vector q and the visible keys j:
//   t_j = scale * (q H / sqrt(D)) . (ks_j kc_j)     w = softmax(t)
//   out = rnd((sum_j w_j vs_j vc_j) H / sqrt(D))    no visible key: 0
// kc, vc the codes of the rotated heads, ks, vs their scales: the rotation
// leaves q . k as it is, so the cache is read as it lies, the query is rotated
// once, and the rotation of the values is taken back once at the end.
//
// A wave's work is a unit of 32 keys against 16 NT query columns, a column
// being one query head of one token: the heads that share a key head, and
// tokens of one sequence, share its unit.  Both products are 16 x 16 matrix
// instructions whose rows are keys, or the values' dims, and whose columns are
// the queries.  The order in which the rows of codes enter gives quarter g of
// the wave the scores of keys 8 g .. 8 g + 7 of its column, which are those that
// the weights' operand has to hold: they go from one product to the next without
// leaving their lane.  The softmax keeps a running reference m and sum l a
// column, in base 2 and fp32.
//
// m is not the maximum of t but of t + log2 vs, what the rounded weight is made
// of, so that fp16 holds it whatever the scales are; it is a whole number, moves
// only where a weight would pass 2^kRise times the last one, and the sums are
// then rescaled by an exact power of two.  A weight times its value's scale is
// rounded to fp16, 11 bits: more than an output of bf16 has; for one of fp16,
// which has as many, it enters as the sum of two (2.1e-4 off, which is the output's
// own rounding, for 2.9e-4 in one; 1 to 12 % of the time where rows are few, 21 % of
// long prompts).  Where one reference is taken for eight keys, or a unit, it is of
// the largest t and the largest vs of them: six powers of two above the largest
// weight at most, for where scales lie further apart keys go one by one.
//
// Few rows (attend_few).  The units come from HBM once and bound the kernel, so
// the codes enter as they lie: scores are int8 products of the codes and of the
// rotated query in two digits of 8 bits, 15 bits together (one fp16, 11 bits,
// was fewer than an fp16 output needs: 4.7e-4 off where 3.1e-4 was reached), with
// the 8 that a code is held with taken off through the sum's first value.  The
// weights' product takes the value codes as fp16: four bits under an exponent
// read as 1024 + u or 1024 + 16 u, and one packed operation makes the code of it,
// without rounding.  A workgroup's four waves take every fourth unit, each with
// its loads one unit ahead, and join their sums in LDS; long sequences are cut
// into parts, joined by a launch of their own.  64 tokens of 64 sequences of up
// to 8192, 32 heads of 128 on 8: 70 us, 4.0 TB/s (5 of it the join); 4 of up to
// 131000, 64 heads on 8: 106 us, 3.3 TB/s (8 the join; vector unit 38 %, matrix unit
// 9 % busy: what is missing is bytes on their way, a unit a wave, 12 waves a CU, and
// parts of even length); 1 of 1000: 11.0 us, latencies one behind the other: table,
// unit, products, the waves' sums.
//
// Many rows (make_operands, attend_many).  A unit then serves hundreds of columns
// and the products and exponentials bound the kernel.  Turning codes into operands
// and scaling scores in every tile cost as much as the products (240 us where 231
// were reached), so one launch before writes keys and values as fp16 operands with
// their scales in them, and the tiles fetch those straight into LDS, two groups of
// units in turn, one worked on while the next is on its way.  A query of bf16 enters
// as one fp16, 11 bits for an output of 8; one of fp16 as the sum of two.  The scores
// of the next unit are started beside the exponentials of this one.  A causal
// prompt of 4608, 32 heads of 128 on 8: 239 us, 727 TFLOP/s counting visible keys
// (9 of it for the operands); three pieces of 667 to 1001 behind up to 16000, 24
// heads of 64, fp16, two terms: 454 us, 400 TFLOP/s (45 for the operands, which is
// their bytes at 6 TB/s).  Matrix and vector unit are busy 30 and 45 %, 38 and 52 %:
// a wave's products and exponentials follow each other, and two waves a SIMD, all
// that the registers hold, cover little of that for each other.
#include <algorithm>

#include "cache.hpp"

namespace convrot {
namespace {

typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

constexpr int kAttnWaves = 4;
constexpr int kAttnThreads = kAttnWaves * 64;
// A column's largest rounded weight lies in [2^kTop, 2^(kTop + kRise)], far
// enough below fp16's 2^16, and one that is 2^-22 of it still has all its bits.
constexpr float kTop = 8.0f;
constexpr float kRise = 6.0f;
// A key that a column does not see; no score is as low.
constexpr float kHidden = -0x1.fffffep127f;
// Value scales below 2^-80 count as that in the reference: the sum l, which has
// no such factor, then stays below 2^(80 + 14) a key.
constexpr int kLeastLevel = -80;
constexpr float kLeastScale = kLeastLevel;
// Value scales that are closer than this share a place in the reference: taken of the largest score
// and the largest scale, it is then six powers of two above the largest weight at most.
constexpr float kSpread = 0x1p-6f;
// Before the first key: below every score, and finite.
constexpr float kNoReference = -0x1p120f;
constexpr float kLog2e = 1.44269504088896340736f;

template <int D> struct RootScale;      // 1 / sqrt(D)
template <> struct RootScale<64> { static constexpr float value = 0.125f; };
template <> struct RootScale<128> { static constexpr float value = 0x1.6a09e6p-4f; };
template <> struct RootScale<256> { static constexpr float value = 0x1p-4f; };

// Rows (16 lanes) of two registers exchanged: of a the odd ones with the even ones of b,
// or the upper two with the lower two.
template <int T>
__device__ inline void swap_rows(float& a, float& b) {
  const auto r = T == 16 ? __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false)
                         : __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  a = __uint_as_float(r[0]);
  b = __uint_as_float(r[1]);
}
// Maximum and sum over the four lanes that share a column.
__device__ inline float column_max(float v) {
  float w = v;
  swap_rows<16>(v, w);
  v = w = fmaxf(v, w);
  swap_rows<32>(v, w);
  return fmaxf(v, w);
}
__device__ inline float column_sum(float v) {
  float w = v;
  swap_rows<16>(v, w);
  v = w = v + w;
  swap_rows<32>(v, w);
  return v + w;
}
__device__ inline int column_sum(int v) {
  auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = static_cast<int>(r[0] + r[1]);
  r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return static_cast<int>(r[0] + r[1]);
}

__device__ inline int wave_index() { return __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6)); }

// The constants of a word's way to fp16, the exponents in a vector register and
// the masks in scalar ones: one instruction then takes both.
struct Spread {
  uint32_t exponent, low, high;
  __device__ Spread() : exponent(0x64006400u), low(0x000f000fu), high(0x00f000f0u) {
    asm volatile("" : "+v"(exponent));
    asm volatile("" : "+s"(low), "+s"(high));
  }
};

// a and b without what a pair of fp16 has of them: one instruction each, which takes an fp16 as it lies.
__device__ inline void take_off(v2h pair, float& a, float& b) {
  asm("v_fma_mix_f32 %0, %1, -1.0, %0 op_sel_hi:[1,0,0]" : "+v"(a) : "v"(pair));
  asm("v_fma_mix_f32 %0, %1, -1.0, %0 op_sel:[1,0,0] op_sel_hi:[1,0,0]" : "+v"(b) : "v"(pair));
}

// Eight codes of a word as fp16, in the order of its nibbles 0 4 1 5 2 6 3 7.
__device__ inline v8h codes_of(uint32_t w, const Spread& c) {
  const v2h off = {static_cast<_Float16>(-1032), static_cast<_Float16>(-1032)};
  const v2h sixteenth = {static_cast<_Float16>(0.0625f), static_cast<_Float16>(0.0625f)};
  const v2h off16 = {static_cast<_Float16>(-72), static_cast<_Float16>(-72)};
  auto low = [&](uint32_t x) { return __builtin_bit_cast(v2h, (x & c.low) | c.exponent) + off; };
  auto high = [&](uint32_t x) {
    return __builtin_elementwise_fma(__builtin_bit_cast(v2h, (x & c.high) | c.exponent), sixteenth, off16);
  };
  const uint32_t w8 = w >> 8;
  const v2h p[4] = {low(w), high(w), low(w8), high(w8)};
  return __builtin_bit_cast(v8h, p);
}

// Sixteen codes of two words as the bytes they are held in (code + 8).
__device__ inline v4i key_codes(uint32_t w0, uint32_t w1) {
  return v4i{static_cast<int>(w0 & 0x0f0f0f0fu), static_cast<int>(w0 >> 4 & 0x0f0f0f0fu),
             static_cast<int>(w1 & 0x0f0f0f0fu), static_cast<int>(w1 >> 4 & 0x0f0f0f0fu)};
}

// What a lane holds of one unit: the words of two tokens' key codes (dims
// [D / 4 * g, D / 4 * (g + 1))), of D / 16 dims' value codes (octet g), and the
// scales of octet g, bf16.
template <int D> struct UnitWords {
  uint32_t k[2][D / 32], v[D / 16];
  uint4 ks, vs;
};

template <int N>
__device__ inline void load_words(const uint8_t* p, uint32_t (&w)[N]) {
  if constexpr (N == 2) {
    const uint2 r = *reinterpret_cast<const uint2*>(p);
    w[0] = r.x, w[1] = r.y;
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 r = reinterpret_cast<const uint4*>(p)[i];
      w[4 * i] = r.x, w[4 * i + 1] = r.y, w[4 * i + 2] = r.z, w[4 * i + 3] = r.w;
    }
  }
}

__device__ inline void widen_scales(const uint4& r, float (&s)[8]) {
  s[0] = bf16_lo(r.x), s[1] = bf16_hi(r.x), s[2] = bf16_lo(r.y), s[3] = bf16_hi(r.y);
  s[4] = bf16_lo(r.z), s[5] = bf16_hi(r.z), s[6] = bf16_lo(r.w), s[7] = bf16_hi(r.w);
}

// One sequence's units of one key head, in the order they are asked for: the
// table's entries are held 64 at a time, one a lane, so that a page's place is
// no load behind a load.
template <int D>
struct UnitReader {
  const Cache& c;
  const int32_t* table;
  int head, held;                       // first table column held
  int32_t entry;

  __device__ UnitReader(const Cache& cache, int b, int h, int column)
      : c(cache), table(cache.table + b * cache.table_stride), head(h) {
    hold(column);
  }
  __device__ void hold(int column) {
    held = column;
    const int at = column + static_cast<int>(threadIdx.x & 63);
    entry = at < (c.max_tokens >> c.page_shift) ? table[at] : -1;
  }

  // A unit; where no page of the cache is named for it another page's, and there = false.
  __device__ __forceinline__ const uint8_t* place(int u, bool& there) {
    const int shift = c.page_shift - 5;
    const int column = u >> shift;
    if (column < held || column >= held + 64) hold(column);
    const int64_t page = __builtin_amdgcn_readlane(entry, column - held);
    there = page >= 0 && page < c.n_pages;
    return c.pages + (there ? page * c.page_bytes : 0) +
           static_cast<int64_t>((head << shift) + (u & ((1 << shift) - 1))) * unit_bytes(D);
  }
  // The key words of tile h and four of the value words.
  static __device__ __forceinline__ void load_keys(const uint8_t* unit, int h, uint32_t (&w)[D / 32]) {
    const int m = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
    load_words(unit + (8 * (m >> 2) + 4 * h + (m & 3)) * (D / 2) + g * (D / 8), w);
  }
  static __device__ __forceinline__ void load_values(const uint8_t* unit, int i, uint32_t (&w)[4]) {
    const int m = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
    load_words(unit + value_codes_at(D) + (g * D + 64 * i + 4 * m) * 4, w);
  }

  __device__ __forceinline__ bool load(int u, UnitWords<D>& w) {
    bool there;
    words(place(u, there), w);
    return there;
  }
  static __device__ __forceinline__ void words(const uint8_t* unit, UnitWords<D>& w) {
    const int g = (threadIdx.x & 63) >> 4;
    load_keys(unit, 0, w.k[0]);
    load_keys(unit, 1, w.k[1]);
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      uint32_t r[4];
      load_values(unit, i, r);
#pragma unroll
      for (int j = 0; j < 4; ++j) w.v[4 * i + j] = r[j];
    }
    w.ks = *reinterpret_cast<const uint4*>(unit + key_scales_at(D) + 16 * g);
    w.vs = *reinterpret_cast<const uint4*>(unit + value_scales_at(D) + 16 * g);
  }
};

// The keys [first, end) that token i of a sequence's rows sees.
__device__ inline void bounds_of(const Attention& a, int64_t start, int length, int i, int& first, int& end) {
  const int64_t pos = start + i;
  end = a.causal ? static_cast<int>(max(int64_t{0}, min(pos + 1, static_cast<int64_t>(length)))) : length;
  first = a.window != 0 ? static_cast<int>(max(int64_t{0}, min(pos + 1 - a.window, int64_t{0x7fffffff}))) : 0;
}

// H_D of a query: five bits of the dim by a product with +-1 (exact, sums in fp32), the
// others, those of the chunk, by sums inside the lane.  A lane has dims [E g, E (g + 1)),
// E = D / 4, as of the keys: in chunk k the eight of bits 0, 1 and the highest of them,
// and out come rows 4 g + i of two tiles, bits 0, 1 and that one.
// The +-1 of row 4 r + i and dims (bits 0, 1, of quarter g): the parity of the bits that
// both have.
template <typename In>
__device__ inline void query_signs(uint32_t (&signs)[2]) {
  constexpr uint32_t kOne = std::is_same_v<In, _Float16> ? 0x3c003c00u : 0x3f803f80u;
  const int col = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
  const uint32_t quarter = __builtin_popcount((col >> 2) & g) & 1 ? 0x80008000u : 0u;
  const uint32_t one = (col & 1) != 0 ? 0x80000000u : 0u, two = (col & 2) != 0 ? 0x80008000u : 0u;
  signs[0] = kOne ^ quarter ^ one;
  signs[1] = signs[0] ^ two;
}
template <int D, typename In, int E = D / 4>
__device__ inline void rotate_query(const uint32_t (&raw)[E / 2], const uint32_t (&signs)[2], float (&v)[E]) {
#pragma unroll
  for (int k = 0; k < E / 8; ++k) {
    const uint32_t in[4] = {raw[2 * k], raw[2 * k + 1], raw[E / 4 + 2 * k], raw[E / 4 + 2 * k + 1]};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t flip = h != 0 ? 0x80008000u : 0u;
      const uint32_t sign[4] = {signs[0], signs[1], signs[0] ^ flip, signs[1] ^ flip};
      const v4f zero = {0.0f, 0.0f, 0.0f, 0.0f};
      v4f r;
      if constexpr (std::is_same_v<In, _Float16>)
        r = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, sign), __builtin_bit_cast(v8h, in), zero, 0, 0, 0);
      else
        r = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, sign), __builtin_bit_cast(v8bf, in), zero, 0, 0, 0);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[E / 2 * h + 4 * k + e] = r[e];
    }
  }
#pragma unroll
  for (int h = 4; h < E / 2; h <<= 1) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      if ((e & h) == 0) {
        const float x = v[e], y = v[e + h];
        v[e] = x + y;
        v[e + h] = x - y;
      }
    }
  }
}

// Rows row0 + 16 t + lane % 16 of a sequence's n * group: their queries' words as they
// lie, and the keys each sees; padding sees everything, so that it never masks a unit.
template <int D, int NT, typename In>
__device__ __forceinline__ void fetch_queries(const Attention& a, int group, int kv_head, int off, int n, int64_t start,
                                              int length, int row0, uint32_t (&raw)[NT][D / 8], int (&from)[NT],
                                              int (&to)[NT]) {
  constexpr int E = D / 4;
  const int col = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4, all = n * group;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int row = row0 + 16 * t + col;
    const bool live = row < all;
    const int i = live ? row / group : 0;
    const int head = kv_head * group + (live ? row - i * group : 0);
    from[t] = 0, to[t] = 0x7fffffff;
    if (live) bounds_of(a, start, length, i, from[t], to[t]);
    const In* p = static_cast<const In*>(a.q) + (static_cast<int64_t>(off) + i) * a.q_stride +
                  static_cast<int64_t>(head) * D + g * E;
#pragma unroll
    for (int j = 0; j < E / 8; ++j) {
      const uint4 r = live ? reinterpret_cast<const uint4*>(p)[j] : make_uint4(0, 0, 0, 0);
      raw[t][4 * j] = r.x, raw[t][4 * j + 1] = r.y, raw[t][4 * j + 2] = r.z, raw[t][4 * j + 3] = r.w;
    }
  }
}

// 16 NT query columns of a wave: their queries, bounds and running sums.  TWO: a weight times
// its value's scale enters as the sum of two fp16.
template <int D, int NT, bool TWO>
struct Columns {
  v4i hi[NT][D / 64], lo[NT][D / 64];   // the queries as 256 hi + lo
  int eight[NT];                        // -8 times a column's sum of them: codes are held as c + 8
  float qs[NT];                         // what one step of them stands for, with |scale| and log2(e)
  int from[NT], to[NT];                 // visible keys of a column
  float m[NT], l[NT];                   // reference; sum of this lane's keys
  v4f o[NT][D / 16];                    // value dims 64 (t / 4) + 16 g + 4 i + t % 4 in o[][t][i]
  int full_from, full_to;               // keys that every column sees
  int any_from, any_to;                 // keys that some column sees

  // Columns of tile rows [row0, row0 + 16 NT) of a sequence's n * group rows; meanwhile()
  // is called while their queries are on the way.
  template <typename In, typename F>
  __device__ __forceinline__ void open(const Attention& a, int group, int kv_head, int off, int n, int64_t start,
                                       int length, int row0, F&& meanwhile) {
    // bounds grow from token to token
    constexpr int E = D / 4;            // dims of a lane
    const int all = n * group;
    bounds_of(a, start, length, row0 / group, any_from, full_to);
    bounds_of(a, start, length, (min(row0 + 16 * NT, all) - 1) / group, full_from, any_to);
    uint32_t signs[2];
    query_signs<In>(signs);
    uint32_t raw[NT][E / 2];
    fetch_queries<D, NT, In>(a, group, kv_head, off, n, start, length, row0, raw, from, to);
    meanwhile();
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float v[E];
      rotate_query<D, In>(raw[t], signs, v);
      float top = 0.0f;
#pragma unroll
      for (int e = 0; e < E; ++e) top = fmaxf(top, fabsf(v[e]));
      top = column_max(top);
      // an infinity or NaN is in every sum of its row; one that only a sum has is in the
      // maximum
      const bool finite = fabsf(v[0]) < __builtin_inff() && top < __builtin_inff();
      // steps of top / 32512, so that both digits fit; the scores of a row that is not
      // finite are NaN by their factor
      const float least = fmaxf(top, 0x1p-100f);
      qs[t] = finite ? least * (RootScale<D>::value * kLog2e / 32512.0f) * fabsf(a.scale) : __builtin_nanf("");
      const float steps = finite ? (a.scale < 0.0f ? -32512.0f : 32512.0f) / least : 0.0f;
      int sum = 0, ones = 0;            // of the digits
#pragma unroll
      for (int k = 0; k < D / 64; ++k) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          // the nearest whole number is in the low bits behind 1.5 * 2^23, its upper digit
          // above them once 128 is added
          uint32_t c[4], c128[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x = finite ? v[16 * k + 8 * (r >> 1) + 2 * e + (r & 1)] : 0.0f;
            const float at = __builtin_fmaf(x, steps, 12582912.0f);
            c[e] = __float_as_uint(at);
            c128[e] = __float_as_uint(at + 128.0f);
          }
          const uint32_t low = __builtin_amdgcn_perm(c[1], c[0], 0x0c0c0400u) | __builtin_amdgcn_perm(c[3], c[2], 0x04000c0cu);
          const uint32_t high =
              __builtin_amdgcn_perm(c128[1], c128[0], 0x0c0c0501u) | __builtin_amdgcn_perm(c128[3], c128[2], 0x05010c0cu);
          hi[t][k][r] = static_cast<int>(high);
          lo[t][k][r] = static_cast<int>(low);
          sum = __builtin_amdgcn_sdot4(static_cast<int>(high), 0x01010101, sum, false);
          ones = __builtin_amdgcn_sdot4(static_cast<int>(low), 0x01010101, ones, false);
        }
      }
      eight[t] = -8 * (256 * column_sum(sum) + column_sum(ones));
      m[t] = kNoReference;
      l[t] = 0.0f;
#pragma unroll
      for (int d = 0; d < D / 16; ++d) o[t][d] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    }
  }

  // One unit; where some column does not see all of it, masked.
  __device__ __forceinline__ void step(const UnitWords<D>& w, const Spread& spread, int u) {
    const int g = (threadIdx.x & 63) >> 4;
    const bool masked = kUnit * u < full_from || kUnit * u + kUnit > full_to;
    float ks[8], vs[8];
    widen_scales(w.ks, ks);
    widen_scales(w.vs, vs);
    float y[NT][8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      v4i key[D / 64];
#pragma unroll
      for (int k = 0; k < D / 64; ++k) key[k] = key_codes(w.k[h][2 * k], w.k[h][2 * k + 1]);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        v4i high = {0, 0, 0, 0}, low = {eight[t], eight[t], eight[t], eight[t]};
#pragma unroll
        for (int k = 0; k < D / 64; ++k) {
          high = __builtin_amdgcn_mfma_i32_16x16x64_i8(key[k], hi[t][k], high, 0, 0, 0);
          low = __builtin_amdgcn_mfma_i32_16x16x64_i8(key[k], lo[t][k], low, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) y[t][4 * h + i] = static_cast<float>((high[i] << 8) + low[i]) * ks[4 * h + i];
      }
    }
    // the reference, kTop below what the largest weight may be made of: the largest score and scale
    // of an octet, or, where those may be far from any one key's, each key's own
    const float large = fmaxf(fmaxf(fmaxf(vs[0], vs[1]), fmaxf(vs[2], vs[3])), fmaxf(fmaxf(vs[4], vs[5]), fmaxf(vs[6], vs[7])));
    const float small = fminf(fminf(fminf(vs[0], vs[1]), fminf(vs[2], vs[3])), fminf(fminf(vs[4], vs[5]), fminf(vs[6], vs[7])));
    float most[NT];
    if (masked || __any(small < large * kSpread)) {
      const int first = kUnit * u + 8 * g;
#pragma unroll
      for (int t = 0; t < NT; ++t) most[t] = kNoReference;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float level = log_scale(vs[i]);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const bool seen = first + i >= from[t] && first + i < to[t];
          y[t][i] = seen ? y[t][i] : kHidden;
          most[t] = fmaxf(most[t], seen ? __builtin_fmaf(y[t][i], qs[t], level) : kNoReference);
        }
      }
    } else {
      const float level = log_scale(large);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float* x = y[t];
        most[t] = __builtin_fmaf(fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7]))),
                                 qs[t], level);
      }
    }
    bool move = false;
#pragma unroll
    for (int t = 0; t < NT; ++t) move = move || most[t] > m[t] + (kTop + kRise);
    if (__any(move)) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        most[t] = column_max(most[t]);
        const float wanted = __builtin_ceilf(most[t]) - kTop;
        if (wanted > m[t] + kRise) {
          const float f = __builtin_amdgcn_exp2f(m[t] - wanted);        // 0 for the first keys
          m[t] = wanted;
          l[t] *= f;
#pragma unroll
          for (int d = 0; d < D / 16; ++d) o[t][d] *= f;
        }
      }
    }
    v8h p[NT], rest[NT];
    auto weights = [&](auto hidden) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float e[8], v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          e[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(y[t][i], qs[t], -m[t]));
          v[i] = e[i] * vs[i];
          if constexpr (hidden.value) {
            // nothing of a key that is not seen, whatever its place holds
            e[i] = y[t][i] == kHidden ? 0.0f : e[i];
            v[i] = y[t][i] == kHidden ? 0.0f : v[i];
          }
        }
        l[t] += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
        v2h pairs[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) pairs[i] = __builtin_convertvector((v2f{v[i], v[i + 4]}), v2h);
        p[t] = __builtin_bit_cast(v8h, pairs);
        if constexpr (TWO) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            pairs[i] = __builtin_convertvector((v2f{v[i] - static_cast<float>(pairs[i][0]), v[i + 4] - static_cast<float>(pairs[i][1])}), v2h);
          rest[t] = __builtin_bit_cast(v8h, pairs);
        }
      }
    };
    if (masked) weights(std::true_type{});
    else weights(std::false_type{});
#pragma unroll
    for (int d = 0; d < D / 16; ++d) {
      const v8h value = codes_of(w.v[d], spread);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        o[t][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(value, p[t], o[t][d], 0, 0, 0);
        if constexpr (TWO) o[t][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(value, rest[t], o[t][d], 0, 0, 0);
      }
    }
  }

  // log2 of a value scale (of NaN the least).
  static __device__ float log_scale(float v) { return fmaxf(__builtin_amdgcn_logf(v), kLeastScale); }

  // Units first, first + by, ... below last, each loaded while the one before is worked on;
  // the first is in a already.
  __device__ __forceinline__ void run(UnitReader<D>& reader, UnitWords<D>& a, bool there_a, int first, int last, int by) {
    if (first >= last) return;
    const Spread spread;
    auto take = [&](const UnitWords<D>& w, int u, bool there) {
      if (there) step(w, spread, u);
    };
    UnitWords<D> b;
    bool there_b = false;
    for (int u = first;;) {
      if (u + by < last) there_b = reader.load(u + by, b);
      take(a, u, there_a);
      u += by;
      if (u >= last) break;
      if (u + by < last) there_a = reader.load(u + by, a);
      take(b, u, there_b);
      u += by;
      if (u >= last) break;
    }
  }
};

// The sums of one column, 16 lanes with E = D / 16 dims each: rotated back, divided
// and rounded.
template <int D, typename In, int E = D / 16>
__device__ inline void finish(float (&v)[E], float l, int part, In* out) {
#pragma unroll
  for (int h = 1; h < E; h <<= 1) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      if ((e & h) == 0) {
        const float x = v[e], y = v[e + h];
        v[e] = x + y;
        v[e + h] = x - y;
      }
    }
  }
  const float by = l != 0.0f ? RootScale<D>::value / l : 0.0f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    float x = v[e], other;
    other = lane_xor<1>(x);
    x = (part & 1) != 0 ? other - x : x + other;
    other = lane_xor<2>(x);
    x = (part & 2) != 0 ? other - x : x + other;
    other = lane_xor<4>(x);
    x = (part & 4) != 0 ? other - x : x + other;
    other = lane_xor<8>(x);
    x = (part & 8) != 0 ? other - x : x + other;
    v[e] = l != 0.0f ? x * by : 0.0f;
  }
  uint32_t w[E / 2];
#pragma unroll
  for (int e = 0; e < E / 2; ++e) w[e] = pack2<In>(v[2 * e], v[2 * e + 1]);
  if constexpr (E == 4) {
    *reinterpret_cast<uint2*>(out + part * E) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int j = 0; j < E / 8; ++j)
      reinterpret_cast<uint4*>(out + part * E)[j] = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
  }
}

// The tile a workgroup has: rows [row0, ...) of sequence b.
struct Tile {
  int b, off, n, row0, start;
  int slot;                             // of the sequences that have tiles, this one's number
};

// Tile `index` of all sequences' tiles of `rows` rows, a sequence's last first
// (of a causal prompt the longest): offsets are looked at 64 sequences at a time,
// one a lane.  Sequences of at most `few` or more than `many` rows have none here.
__device__ inline bool find_tile(const Attention& a, int group, int rows, int few, int many, int index, Tile& tile) {
  const int lane = threadIdx.x & 63;
  int before = 0, slots = 0;
  for (int b0 = 0; b0 < a.cache.n_seqs; b0 += 64) {
    const int b = b0 + lane;
    Span s{0, 0};
    int start = 0;
    if (b < a.cache.n_seqs) {
      s = span_of(a.offsets, b, a.M);
      start = a.starts[b];
    }
    const int64_t all = static_cast<int64_t>(s.end - s.off) * group;
    const int mine = all > few && all <= many ? static_cast<int>((all + rows - 1) / rows) : 0;
    int sum = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int other = __shfl_up(sum, d);
      if (lane >= d) sum += other;
    }
    const int total = __builtin_amdgcn_readlane(sum, 63);
    if (index - before < total) {
      const uint64_t behind = __ballot(index - before < sum);
      const int l = __builtin_ctzll(behind);
      tile.b = b0 + l;
      tile.slot = slots + __builtin_popcountll(__ballot(mine > 0) & ((uint64_t{1} << l) - 1));
      tile.off = __builtin_amdgcn_readlane(s.off, l);
      tile.n = __builtin_amdgcn_readlane(s.end, l) - tile.off;
      tile.start = __builtin_amdgcn_readlane(start, l);
      const int at = index - before - (__builtin_amdgcn_readlane(sum, l) - __builtin_amdgcn_readlane(mine, l));
      tile.row0 = (__builtin_amdgcn_readlane(mine, l) - 1 - at) * rows;
      return true;
    }
    before += total;
    slots += __builtin_popcountll(__ballot(mine > 0));
  }
  return false;
}

// The keys of a sequence that there are.
__device__ inline int length_of(const Attention& a, const Tile& tile) {
  return static_cast<int>(max(int64_t{0}, min(static_cast<int64_t>(tile.start) + tile.n, static_cast<int64_t>(a.cache.max_tokens))));
}

// A staged unit: the operands of both products, and what goes with them.
template <int D> struct StagedUnit {
  static constexpr int kKeys = 2 * (D / 32), kPieces = kKeys + D / 16;
  const uint4* piece;                   // [kPieces][64]: a lane's 16 bytes of each
  __device__ v8h key(int h, int k) const {
    return __builtin_bit_cast(v8h, piece[(h * (D / 32) + k) * 64 + (threadIdx.x & 63)]);
  }
  __device__ v8h value(int d) const { return __builtin_bit_cast(v8h, piece[(kKeys + d) * 64 + (threadIdx.x & 63)]); }
};
constexpr int kNoScale = -1000;
constexpr float kMostPower = 0x1p126f;  // its reciprocal is normal
constexpr uint32_t kHeld = 1, kUneven = 2;
struct UnitFacts {
  float key;                            // what a 1 of the key operand stands for
  int value;                            // and of the value operand, as its logarithm; kNoScale: all are 0
  uint32_t bad;                         // tokens whose value is not finite
  uint32_t flags;                       // kHeld: a page holds the unit.  kUneven: its tokens' scales are
                                        // far apart, and each has a power of two of its own (Levels)
};
// How far below the unit's a token's power of two is, a byte a token, eight of each kind a lane.
constexpr uint32_t kNothing = 255;      // a value of 0
struct Levels {
  uint32_t key[2], value[2];
  static __device__ __forceinline__ uint32_t of(const uint32_t (&w)[2], int i) { return w[i >> 2] >> (8 * (i & 3)) & 255; }
};

// The state of 16 NT query columns of a wave whose keys and values come as operands
// with their scales in them (Staged): TERMS fp16 values that add up to each of the
// query's, so that a score is the product itself.
template <int D, int NT, int TERMS>
struct PromptColumns {
  v8h q[NT][TERMS][D / 32];
  float qs[NT];                         // what one of them stands for, with |scale| and log2(e)
  int from[NT], to[NT];                 // visible keys of a column
  float m[NT], l[NT];                   // reference; sum of this lane's keys
  v4f o[NT][D / 16];                    // value dims 64 (t / 4) + 16 g + 4 i + t % 4 in o[][t][i]
  int full_from, full_to;               // keys that every column sees
  int any_from, any_to;                 // keys that some column sees

  template <typename In, typename F>
  __device__ __forceinline__ void open(const Attention& a, int group, int kv_head, int off, int n, int64_t start,
                                       int length, int row0, F&& meanwhile) {
    constexpr int E = D / 4;
    const int all = n * group;
    bounds_of(a, start, length, row0 / group, any_from, full_to);
    bounds_of(a, start, length, (min(row0 + 16 * NT, all) - 1) / group, full_from, any_to);
    uint32_t raw[NT][E / 2], signs[2];
    fetch_queries<D, NT, In>(a, group, kv_head, off, n, start, length, row0, raw, from, to);
    meanwhile();
    query_signs<In>(signs);
    const float unit = RootScale<D>::value * kLog2e * fabsf(a.scale);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float v[E];
      rotate_query<D, In>(raw[t], signs, v);
      float top = 0.0f;
#pragma unroll
      for (int e = 0; e < E; ++e) top = fmaxf(top, fabsf(v[e]));
      top = column_max(top);
      const bool finite = fabsf(v[0]) < __builtin_inff() && top < __builtin_inff();
      // the row's largest value to [256, 512): what fp16 does not hold in full is then
      // below 2^-22 of it, in one term or in the second
      const int down = finite ? ilogbf(fmaxf(top, 0x1p-100f)) - 8 : 0;
      const float by = finite ? ldexpf(a.scale < 0.0f ? -1.0f : 1.0f, -down) : 0.0f;
      qs[t] = finite ? ldexpf(unit, down) : __builtin_nanf("");
#pragma unroll
      for (int k = 0; k < D / 32; ++k) {
        constexpr int kOrder[8] = {0, 4, 1, 5, 2, 6, 3, 7};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float x = finite ? v[8 * k + kOrder[e]] * by : 0.0f;
          q[t][0][k][e] = static_cast<_Float16>(x);
          if constexpr (TERMS == 2) q[t][1][k][e] = static_cast<_Float16>(x - static_cast<float>(q[t][0][k][e]));
        }
      }
      m[t] = kNoReference;
      l[t] = 0.0f;
#pragma unroll
      for (int d = 0; d < D / 16; ++d) o[t][d] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    }
  }

  // Scores of a staged unit, in units of qs times the unit's key factor.
  __device__ __forceinline__ void scores(const StagedUnit<D>& unit, v4f (&s)[NT][2]) const {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int t = 0; t < NT; ++t) s[t][h] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int k = 0; k < D / 32; ++k) {
        const v8h key = unit.key(h, k);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int r = 0; r < TERMS; ++r) s[t][h] = __builtin_amdgcn_mfma_f32_16x16x32_f16(key, q[t][r][k], s[t][h], 0, 0, 0);
      }
    }
  }

  // Hides what a column does not see.
  __device__ __forceinline__ void hide(v4f (&s)[NT][2], int u, const UnitFacts& facts) {
    const int first = kUnit * u + 8 * static_cast<int>((threadIdx.x & 63) >> 4);
    const bool held = (facts.flags & kHeld) != 0;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        s[t][i >> 2][i & 3] = held && first + i >= from[t] && first + i < to[t] ? s[t][i >> 2][i & 3] : kHidden;
    if (facts.bad != 0) {
      // a value that is not finite: it is not in the product (there it would reach those
      // who do not see it), but in the sum of who sees it
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if ((facts.bad >> ((first + i) & 31) & 1) != 0 && s[t][i >> 2][i & 3] != kHidden) l[t] = __builtin_nanf("");
    }
  }

  // The logarithm of value i's power of two.
  static __device__ __forceinline__ int level_of(const UnitFacts& facts, const Levels& levels, int i) {
    const uint32_t down = Levels::of(levels.value, i);
    return down == kNothing ? kNoScale : facts.value - static_cast<int>(down);
  }

  // The weights times their values' powers of two.
  __device__ __forceinline__ void weights(const v4f (&s)[NT][2], const float (&f)[NT], const UnitFacts& facts,
                                          const Levels& levels, v8h (&p)[NT][TERMS]) {
    v2h pairs[NT][TERMS][4];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int level = level_of(facts, levels, i), counted = level == kNoScale ? 0 : level;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float x = s[t][i >> 2][i & 3];
        float e = __builtin_amdgcn_exp2f(__builtin_fmaf(x, f[t], static_cast<float>(counted) - m[t]));
        e = x == kHidden ? 0.0f : e;
        l[t] += ldexpf(e, -counted);
        float w = level == kNoScale ? 0.0f : e;
#pragma unroll
        for (int r = 0; r < TERMS; ++r) {
          const auto part = static_cast<_Float16>(w);
          pairs[t][r][i & 3][i >> 2] = part;
          w -= static_cast<float>(part);
        }
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int r = 0; r < TERMS; ++r) p[t][r] = __builtin_bit_cast(v8h, pairs[t][r]);
  }

  __device__ __forceinline__ void add(const StagedUnit<D>& unit, const v8h (&p)[NT][TERMS]) {
#pragma unroll
    for (int d = 0; d < D / 16; ++d) {
      const v8h value = unit.value(d);
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int r = 0; r < TERMS; ++r) o[t][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(value, p[t][r], o[t][d], 0, 0, 0);
    }
  }

  // The references to kTop below `most`, the logarithm of the largest weight times its value's
  // power of two, where one would get too large.
  __device__ __forceinline__ void raise(float (&most)[NT]) {
    bool move = false;
#pragma unroll
    for (int t = 0; t < NT; ++t) move = move || most[t] > m[t] + (kTop + kRise);
    if (__any(move)) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        most[t] = column_max(most[t]);
        const float wanted = __builtin_ceilf(most[t]) - kTop;
        if (wanted > m[t] + kRise) {
          const float down = __builtin_amdgcn_exp2f(m[t] - wanted);     // 0 for the first keys
          m[t] = wanted;
          l[t] *= down;
#pragma unroll
          for (int d = 0; d < D / 16; ++d) o[t][d] *= down;
        }
      }
    }
  }
  // What it takes of the keys that a column sees, one by one: the mark of a hidden one is no score
  // (times the unit's factor, 0 where no page or no key holds anything, it would be one).
  __device__ __forceinline__ void raise_seen(const v4f (&s)[NT][2], const float (&f)[NT], const UnitFacts& facts,
                                             const Levels& levels) {
    float most[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) most[t] = kNoReference;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float level = static_cast<float>(max(level_of(facts, levels, i), kLeastLevel));
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float x = s[t][i >> 2][i & 3];
        most[t] = __builtin_elementwise_maximum(most[t], x == kHidden ? kNoReference : __builtin_fmaf(x, f[t], level));
      }
    }
    raise(most);
  }
  // (NaN if one is: no canonical form is made of its operands first)
  static __device__ __forceinline__ float max3(float a, float b, float c) {
    return __builtin_elementwise_maximum(__builtin_elementwise_maximum(a, b), c);
  }

  // A whole group that every column sees all of, its units even.
  template <int UNITS, typename Group>
  __device__ __forceinline__ void whole_group(const Group& group) {
    v4f s[NT][2];
    scores(group.unit(0), s);
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
      const int value = group.value(i);
      const float level = static_cast<float>(value);
      float f[NT], most[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const v4f a = s[t][0], b = s[t][1];
        f[t] = qs[t] * group.key(i);
        most[t] = __builtin_fmaf(max3(max3(max3(a[0], a[1], a[2]), a[3], b[0]), max3(b[1], b[2], b[3]), b[3]), f[t], level);
      }
      raise(most);
      v8h p[NT][TERMS];
      v4f next[NT][2];
      if (i + 1 < UNITS) scores(group.unit(i + 1), next);
      const float back = __uint_as_float(static_cast<uint32_t>(127 - value) << 23);   // 2^-value
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float low = level - m[t];
        float e[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) e[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][j >> 2][j & 3], f[t], low));
        l[t] = __builtin_fmaf(((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7])), back, l[t]);
#pragma unroll
        for (int r = 0; r < TERMS; ++r) {
          v2h pairs[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            pairs[j] = __builtin_convertvector((v2f{e[j], e[j + 4]}), v2h);
            if (r + 1 < TERMS) take_off(pairs[j], e[j], e[j + 4]);
          }
          p[t][r] = __builtin_bit_cast(v8h, pairs);
        }
      }
      add(group.unit(i), p);
#pragma unroll
      for (int t = 0; t < NT; ++t) s[t][0] = next[t][0], s[t][1] = next[t][1];
    }
  }

  // Units [i0, i1) of a staged group, where something is hidden or not as usual; levels_of(i)
  // where a unit's scales are far apart.
  template <typename Group, typename F>
  __device__ __forceinline__ void steps(const Group& group, int u0, int i0, int i1, F&& levels_of) {
#pragma unroll 1
    for (int i = i0; i < i1; ++i) {
      const UnitFacts facts = group.facts(i);
      const uint32_t down = facts.value == kNoScale ? ~0u : 0u;
      Levels levels{{0, 0}, {down, down}};
      float f[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) f[t] = qs[t] * facts.key;
      v4f s[NT][2];
      v8h p[NT][TERMS];
      scores(group.unit(i), s);
      if ((facts.flags & kUneven) != 0) {
        levels = levels_of(u0 + i);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int by = -static_cast<int>(Levels::of(levels.key, k));
#pragma unroll
          for (int t = 0; t < NT; ++t) s[t][k >> 2][k & 3] = ldexpf(s[t][k >> 2][k & 3], by);
        }
      }
      hide(s, u0 + i, facts);
      raise_seen(s, f, facts, levels);
      weights(s, f, facts, levels, p);
      add(group.unit(i), p);
    }
  }
};

// The power of two at or below a scale; 0 for what has none that is normal.
__device__ inline float power_below(float v) { return __uint_as_float(__float_as_uint(v) & 0x7f800000u); }

// A long prompt's keys and values as the operands of both products, made once in the
// workspace for all of its tiles: [slot][key head][unit] of kPieces KB, and behind them the
// facts of as many units, and their levels.  A code times its scale is exact in fp16, 3 bits by
// 8, the scales taken relative to a power of two of their unit; where some lie more than kSpread
// below the largest, each relative to one of its own.
template <int D>
struct Operands {
  static constexpr int kPieces = StagedUnit<D>::kPieces, kKeys = StagedUnit<D>::kKeys;
  uint4* piece;
  UnitFacts* facts;
  uint8_t* levels;                      // [unit][64]: keys, values
  __device__ Operands(const Attention& a, int slot, int head) {
    const int64_t all = static_cast<int64_t>(a.slots) * a.cache.kv_heads * a.slot_units;
    const int64_t at = (static_cast<int64_t>(slot) * a.cache.kv_heads + head) * a.slot_units;
    piece = reinterpret_cast<uint4*>(a.operands) + at * (kPieces * 64);
    facts = reinterpret_cast<UnitFacts*>(a.operands + all * (kPieces * 1024)) + at;
    levels = a.operands + all * (kPieces * 1024 + static_cast<int64_t>(sizeof(UnitFacts))) + at * 64;
  }
  __device__ Levels levels_of(int u) const {
    const uint8_t* p = levels + static_cast<int64_t>(u) * 64 + 8 * ((threadIdx.x & 63) >> 4);
    const uint2 k = *reinterpret_cast<const uint2*>(p), v = *reinterpret_cast<const uint2*>(p + 32);
    return Levels{{k.x, k.y}, {v.x, v.y}};
  }
};

// One unit a wave: what it reads comes once, and what it writes bounds it (24 heads of 64,
// 34000 tokens: 45 us, 5.9 TB/s).
template <int D>
__global__ __launch_bounds__(kAttnThreads) void make_operands(Attention a, int few) {
  using O = Operands<D>;
  __shared__ alignas(16) _Float16 scales[kAttnWaves][64];
  const int lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4, wave = wave_index();
  const int u = static_cast<int>(blockIdx.x) * kAttnWaves + wave, head = static_cast<int>(blockIdx.y);
  Tile tile;
  if (!find_tile(a, a.q_heads / a.cache.kv_heads, 0x40000000, few, 0x7fffffff, static_cast<int>(blockIdx.z), tile)) return;
  const int length = length_of(a, tile);
  int seen, unused;                     // from the first row's first key on
  bounds_of(a, tile.start, length, 0, seen, unused);
  if (kUnit * u >= length || kUnit * (u + 1) <= seen) return;
  const O out(a, tile.slot, head);
  UnitReader<D> reader(a.cache, tile.b, head, u >> (a.cache.page_shift - 5));
  bool held;
  const uint8_t* unit = reader.place(u, held);
  UnitWords<D> w;
  reader.words(unit, w);
  const uint32_t bits = reinterpret_cast<const uint16_t*>(unit + key_scales_at(D))[lane];
  const Spread spread;
  // the scale of key lane, or of value lane - 32; of places behind the last token nothing
  float scale = held && kUnit * u + (lane & 31) < length ? __uint_as_float(bits << 16) : 0.0f;
  const bool finite = fabsf(scale) < __builtin_inff();
  const uint64_t broken = __ballot(!finite);
  const float own = finite ? power_below(scale) : 0.0f;
  float top = own;
  top = fmaxf(top, lane_xor<1>(top));
  top = fmaxf(top, lane_xor<2>(top));
  top = fmaxf(top, lane_xor<4>(top));
  top = fmaxf(top, lane_xor<8>(top));
  float other = top;
  swap_rows<16>(top, other);
  top = fminf(fmaxf(top, other), kMostPower);
  // keys by what fp16 holds of the small ones (none is lost where they are 0), values by how far the
  // references may be above the weights of one that they are taken of
  const bool is_key = lane < 32, there = held && finite && kUnit * u + (lane & 31) < length;
  const bool uneven = __any(there && (is_key ? own > 0.0f && own < top * 0x1p-14f : own < top * kSpread));
  if (!finite && !is_key) scale = 0.0f;
  const float unit_of = uneven && own > 0.0f ? fminf(own, kMostPower) : top;
  scales[wave][lane] = static_cast<_Float16>(unit_of > 0.0f ? scale * (1.0f / unit_of) : scale * 0.0f);
  if (uneven) {
    const uint32_t down = (__float_as_uint(top) - __float_as_uint(unit_of)) >> 23;
    out.levels[static_cast<int64_t>(u) * 64 + lane] = static_cast<uint8_t>(own > 0.0f || is_key ? down : kNothing);
  }
  const float key = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(top), 0));
  const int value = static_cast<int>(__builtin_amdgcn_readlane(__float_as_uint(top), 32) >> 23);
  if (lane == 0)
    out.facts[u] = UnitFacts{key, value != 0 ? value - 127 : kNoScale, static_cast<uint32_t>(broken >> 32),
                             (held ? kHeld : 0) | (uneven ? kUneven : 0)};
  // lanes of this wave only read what it wrote itself: its writes have to be done, no barrier is due
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  uint4* to = out.piece + static_cast<int64_t>(u) * (O::kPieces * 64) + lane;
  auto store = [&](int i, uint32_t word, const v2h (&by)[4]) {
    const v8h v = codes_of(word, spread);
    v2h p[4];
    __builtin_memcpy(p, &v, sizeof v);
#pragma unroll
    for (int e = 0; e < 4; ++e) p[e] *= by[e];
    to[64 * i] = __builtin_bit_cast(uint4, p);
  };
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const _Float16 by = scales[wave][8 * (m >> 2) + 4 * h + (m & 3)];
    const v2h all[4] = {{by, by}, {by, by}, {by, by}, {by, by}};
#pragma unroll
    for (int k = 0; k < D / 32; ++k) store(h * (D / 32) + k, w.k[h][k], all);
  }
  uint4 eight;
  __builtin_memcpy(&eight, __builtin_assume_aligned(&scales[wave][32 + 8 * g], 16), sizeof eight);
  // the scales of tokens 0 and 4, 1 and 5, 2 and 6, 3 and 7 of the octet
  const uint32_t by_token[4] = {__builtin_amdgcn_perm(eight.z, eight.x, 0x05040100u),
                                __builtin_amdgcn_perm(eight.z, eight.x, 0x07060302u),
                                __builtin_amdgcn_perm(eight.w, eight.y, 0x05040100u),
                                __builtin_amdgcn_perm(eight.w, eight.y, 0x07060302u)};
  v2h all[4];
  __builtin_memcpy(all, by_token, sizeof all);
#pragma unroll
  for (int d = 0; d < D / 16; ++d) store(O::kKeys + d, w.v[d], all);
}

// A group of units in LDS for all waves of a workgroup, whose columns are their own; the
// next group comes straight into the other half while this one is worked on.
template <int D, int WAVES>
struct Staged {
  static constexpr int kUnits = 64 * WAVES / D;                  // a group: a half has 8 KB for each wave
  static constexpr int kPieces = StagedUnit<D>::kPieces, kMine = kUnits * kPieces / WAVES;
  uint4 piece[2][kUnits][kPieces][64];

  struct Group {
    const Staged& s;
    int which;
    UnitFacts of;                       // unit lane % kUnits
    __device__ StagedUnit<D> unit(int i) const { return StagedUnit<D>{&s.piece[which][i][0][0]}; }
    __device__ int value(int i) const { return __builtin_amdgcn_readlane(of.value, i); }
    __device__ float key(int i) const { return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(of.key), i)); }
    __device__ UnitFacts facts(int i) const {
      auto one = [i](uint32_t v) { return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), i)); };
      return UnitFacts{__uint_as_float(one(__float_as_uint(of.key))), static_cast<int>(one(static_cast<uint32_t>(of.value))),
                       one(of.bad), one(of.flags)};
    }
  };

  // This wave's pieces of the group from unit u0 on; those behind a slot's last unit are
  // the slot's own spare ones, or the next slot's first.
  __device__ __forceinline__ void fetch(const Operands<D>& from, int which, int u0) {
    const int at = wave_index() * kMine;
    const uint4* src = from.piece + (static_cast<int64_t>(u0) * kPieces + at) * 64 + (threadIdx.x & 63);
    uint4* dst = &piece[which][0][0][0] + at * 64;
#pragma unroll
    for (int j = 0; j < kMine; ++j)
      __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(src + 64 * j),
                                       (__attribute__((address_space(3))) void*)(dst + 64 * j), 16, 0, 0);
  }
  static __device__ __forceinline__ UnitFacts facts_of(const Operands<D>& from, int u0) {
    return from.facts[u0 + static_cast<int>(threadIdx.x & (kUnits - 1))];
  }

  template <typename Columns>
  __device__ __forceinline__ void run(Columns& c, const Operands<D>& from, const UnitFacts& first_facts, int first, int last,
                                      bool idle) {
    if (first >= last) return;
    UnitFacts facts = first_facts;
    int which = 0;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    for (int u0 = first; u0 < last; u0 += kUnits, which ^= 1) {
      // into the half that all waves were done with before the last barrier
      UnitFacts next = facts;
      if (u0 + kUnits < last) {
        fetch(from, which ^ 1, u0 + kUnits);
        next = facts_of(from, u0 + kUnits);
      }
      const int i0 = max(0, c.any_from / kUnit - u0);
      const int i1 = idle ? 0 : min(min(kUnits, last - u0), (c.any_to + kUnit - 1) / kUnit - u0);
      const Group group{*this, which, facts};
      const bool usual = facts.flags == kHeld && facts.bad == 0 && facts.value >= kLeastLevel;
      if (i0 == 0 && i1 == kUnits && kUnit * u0 >= c.full_from && kUnit * (u0 + kUnits) <= c.full_to && __all(usual))
        c.template whole_group<kUnits>(group);
      else
        c.steps(group, u0, i0, i1, [&](int u) { return from.levels_of(u); });
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();
      facts = next;
    }
  }
};

// Sums over a query's parts: what a workgroup knows of where its rows go.
struct Rows {
  int off, group, kv_head, q_heads;
  // the row of the output (and of a part's sums) that row `row` of a sequence's is
  __device__ int64_t operator()(int row) const {
    const int i = row / group;
    return (static_cast<int64_t>(off) + i) * q_heads + kv_head * group + (row - i * group);
  }
};

// The units [first, last) of a tile's rows [row0, row0 + rows) that belong to a part; the
// parts begin at the first unit that the tile sees.
__device__ inline void units_of(const Attention& a, const Tile& tile, int group, int rows, int part, int64_t start, int length,
                                int& first, int& last) {
  int from, end, unused;
  bounds_of(a, start, length, tile.row0 / group, from, unused);
  bounds_of(a, start, length, (min(tile.row0 + rows, tile.n * group) - 1) / group, unused, end);
  const int64_t base = from / kUnit * kUnit + static_cast<int64_t>(part) * a.chunk;
  const int64_t lo = max(static_cast<int64_t>(from), base);
  const int64_t hi = part == a.splits - 1 ? end : min(static_cast<int64_t>(end), base + a.chunk);
  first = static_cast<int>(min(lo, int64_t{0x7fffffff}) / kUnit);
  last = lo < hi ? static_cast<int>((hi + kUnit - 1) / kUnit) : 0;
}

// Few rows: the four waves have the same 16 NT columns and every fourth unit each.
template <int D, int NT, typename In>
__global__ __launch_bounds__(kAttnThreads, D * NT <= 64 ? 4 : D * NT <= 128 ? 3 : D * NT <= 256 ? 2 : 1) void attend_few(
    Attention a, int few, int many) {
  constexpr int kRows = 16 * NT;
  const int kv_heads = a.cache.kv_heads, group = a.q_heads / kv_heads;
  const int kv_head = static_cast<int>(blockIdx.x % static_cast<unsigned>(kv_heads));
  const int part = static_cast<int>(blockIdx.y);
  Tile tile;
  if (!find_tile(a, group, kRows, few, many, static_cast<int>(blockIdx.x / static_cast<unsigned>(kv_heads)), tile)) return;
  const int wave = wave_index(), lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
  const int length = length_of(a, tile), all = tile.n * group;
  int first, last;
  units_of(a, tile, group, kRows, part, tile.start, length, first, last);
  UnitReader<D> reader(a.cache, tile.b, kv_head, first >> (a.cache.page_shift - 5));
  Columns<D, NT, std::is_same_v<In, _Float16>> c;
  UnitWords<D> words;
  bool there = false;
  c.template open<In>(a, group, kv_head, tile.off, tile.n, tile.start, length, tile.row0,
                      [&] { there = first + wave < last && reader.load(first + wave, words); });
  c.run(reader, words, there, first + wave, last, kAttnWaves);

  const Rows row_of{tile.off, group, kv_head, a.q_heads};
  const int64_t rows = static_cast<int64_t>(a.M) * a.q_heads;
#pragma unroll
  for (int t = 0; t < NT; ++t) c.l[t] = column_sum(c.l[t]);
  constexpr int kStride = D + 4;
  __shared__ alignas(16) float sums[kAttnWaves][16][kStride];
  __shared__ float refs[kAttnWaves][16], totals[kAttnWaves][16];
  const int mine = threadIdx.x >> 4, piece = threadIdx.x & 15;
  constexpr int E = D / 16;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    if (t > 0) __syncthreads();
#pragma unroll
    for (int d = 0; d < D / 64; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<float4*>(&sums[wave][col][64 * d + 16 * g + 4 * i]) =
            make_float4(c.o[t][4 * d][i], c.o[t][4 * d + 1][i], c.o[t][4 * d + 2][i], c.o[t][4 * d + 3][i]);
    if (g == 0) {
      refs[wave][col] = c.m[t];
      totals[wave][col] = c.l[t];
    }
    __syncthreads();
    const int row = tile.row0 + 16 * t + mine;
    float m = refs[0][mine];
#pragma unroll
    for (int w = 1; w < kAttnWaves; ++w) m = fmaxf(m, refs[w][mine]);
    float v[E], l = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = 0.0f;
#pragma unroll
    for (int w = 0; w < kAttnWaves; ++w) {
      const float r = refs[w][mine];
      const float f = __builtin_amdgcn_exp2f(r - m);
      l = __builtin_fmaf(totals[w][mine], f, l);
#pragma unroll
      for (int e = 0; e < E; e += 4) {
        const float4 x = *reinterpret_cast<const float4*>(&sums[w][mine][piece * E + e]);
        v[e] = __builtin_fmaf(x.x, f, v[e]);
        v[e + 1] = __builtin_fmaf(x.y, f, v[e + 1]);
        v[e + 2] = __builtin_fmaf(x.z, f, v[e + 2]);
        v[e + 3] = __builtin_fmaf(x.w, f, v[e + 3]);
      }
    }
    if (row < all) {
      if (a.splits == 1) {
        finish<D, In>(v, l, piece, static_cast<In*>(a.out) + row_of(row) * D);
      } else {
        const int64_t at = part * rows + row_of(row);
        float* to = a.part + at * D + piece * E;
#pragma unroll
        for (int e = 0; e < E; e += 4) *reinterpret_cast<float4*>(to + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
        if (piece == 0)
          *reinterpret_cast<float2*>(a.part + a.splits * rows * D + 2 * at) = make_float2(m, l);
      }
    }
  }
}

// Many rows: the waves have 16 NT columns each and the same units, staged.
template <int D, int NT, int WAVES, typename In>
__global__ __launch_bounds__(64 * WAVES, 2) void attend_many(Attention a, int few, int many) {
  constexpr int kRows = 16 * NT * WAVES;
  const int kv_heads = a.cache.kv_heads, group = a.q_heads / kv_heads;
  const int kv_head = static_cast<int>(blockIdx.x % static_cast<unsigned>(kv_heads));
  const int part = static_cast<int>(blockIdx.y);
  Tile tile;
  if (!find_tile(a, group, kRows, few, many, static_cast<int>(blockIdx.x / static_cast<unsigned>(kv_heads)), tile)) return;
  // as many slots as rows allow: more long prompts are of offsets that rise and fall
  if (tile.slot >= a.slots) return;
  const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
  const int length = length_of(a, tile), all = tile.n * group;
  const int row0 = tile.row0 + 16 * NT * wave_index();
  const bool idle = row0 >= all;        // a wave behind the tile's rows: it only fetches
  int first, last;
  units_of(a, tile, group, kRows, part, tile.start, length, first, last);
  const Operands<D> from(a, tile.slot, kv_head);
  __shared__ Staged<D, WAVES> staged;
  PromptColumns<D, NT, std::is_same_v<In, _Float16> ? 2 : 1> c;
  UnitFacts facts{};
  c.template open<In>(a, group, kv_head, tile.off, tile.n, tile.start, length, idle ? tile.row0 : row0, [&] {
    if (first < last) {
      staged.fetch(from, 0, first);
      facts = staged.facts_of(from, first);
    }
  });
  staged.run(c, from, facts, first, last, idle);
  if (idle) return;

  const Rows row_of{tile.off, group, kv_head, a.q_heads};
  const int64_t rows = static_cast<int64_t>(a.M) * a.q_heads;
#pragma unroll
  for (int t = 0; t < NT; ++t) c.l[t] = column_sum(c.l[t]);
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int row = row0 + 16 * t + col;
    // dims 64 d + 16 g + e of this column
    float v[D / 64][16];
#pragma unroll
    for (int d = 0; d < D / 64; ++d)
#pragma unroll
      for (int e = 0; e < 16; ++e) v[d][e] = c.o[t][4 * d + (e & 3)][e >> 2];
    if (a.splits != 1) {
      if (row < all) {
        const int64_t at = part * rows + row_of(row);
#pragma unroll
        for (int d = 0; d < D / 64; ++d)
#pragma unroll
          for (int e = 0; e < 16; e += 4)
            *reinterpret_cast<float4*>(a.part + at * D + 64 * d + 16 * g + e) =
                make_float4(v[d][e], v[d][e + 1], v[d][e + 2], v[d][e + 3]);
        if (g == 0) *reinterpret_cast<float2*>(a.part + a.splits * rows * D + 2 * at) = make_float2(c.m[t], c.l[t]);
      }
      continue;
    }
    // H_D: bits 0 to 3 of the dim and those from 6 on lie inside a lane; bits 4 and 5
    // are the lane's quarter, which is exchanged with two others of the lane's own, so
    // that each sum has both its terms in one lane: bit 3, and bit 6 (D = 64: bit 2)
#pragma unroll
    for (int d = 0; d < D / 64; ++d) {
#pragma unroll
      for (int h = 1; h < 16; h <<= 1) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          if ((e & h) == 0) {
            const float x = v[d][e], y = v[d][e + h];
            v[d][e] = x + y;
            v[d][e + h] = x - y;
          }
        }
      }
    }
#pragma unroll
    for (int h = 1; h < D / 64; h <<= 1) {
#pragma unroll
      for (int d = 0; d < D / 64; ++d) {
        if ((d & h) == 0) {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float x = v[d][e], y = v[d + h][e];
            v[d][e] = x + y;
            v[d + h][e] = x - y;
          }
        }
      }
    }
#pragma unroll
    for (int d = 0; d < D / 64; ++d) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        swap_rows<16>(v[d][e], v[d][e + 8]);
        const float x = v[d][e], y = v[d][e + 8];
        v[d][e] = x + y;
        v[d][e + 8] = x - y;
      }
    }
    // now bit 3 of the dim is bit 0 of the quarter, and index 8 of a lane bit 4
    auto last = [&](float& p, float& q) {
      swap_rows<32>(p, q);
      const float x = p, y = q;
      p = x + y;
      q = x - y;
    };
    if constexpr (D == 64) {
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if ((e & 4) == 0) last(v[0][e], v[0][e + 4]);
    } else {
#pragma unroll
      for (int d = 0; d < D / 64; d += 2)
#pragma unroll
        for (int e = 0; e < 16; ++e) last(v[d][e], v[d + 1][e]);
    }
    const float by = c.l[t] != 0.0f ? RootScale<D>::value / c.l[t] : 0.0f;
    if (row < all) {
      In* out = static_cast<In*>(a.out) + row_of(row) * D + 8 * (g & 1);
#pragma unroll
      for (int d = 0; d < D / 64; ++d) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float f[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = c.l[t] != 0.0f ? v[d][8 * j + e] * by : 0.0f;
          if constexpr (D == 64) {
            // index 4 of a lane is bit 5, the quarter's bit 1 is bit 2
            const uint4 w = narrow8<In>(f);
            *reinterpret_cast<uint2*>(out + 16 * j + 4 * (g >> 1)) = make_uint2(w.x, w.y);
            *reinterpret_cast<uint2*>(out + 16 * j + 32 + 4 * (g >> 1)) = make_uint2(w.z, w.w);
          } else {
            // d's bit 0 is bit 5, the quarter's bit 1 is bit 6
            *reinterpret_cast<uint4*>(out + 128 * (d >> 1) + 64 * (g >> 1) + 32 * (d & 1) + 16 * j) = narrow8<In>(f);
          }
        }
      }
    }
  }
}

// The parts of a row joined, a wave a row: first every part's reference and sum, a
// part a lane, then four parts at a time by 16 lanes each.  Parts whose keys the row
// does not see hold nothing of it and are not read.  64 rows of 32 heads in three parts:
// 4.8 us, a launch's length; 4 of 64 in 43 parts: 8.0.
template <int D, typename In>
__global__ __launch_bounds__(kAttnThreads) void join_kernel(Attention a, int few_rows, int many, int many_rows) {
  constexpr int E = D / 16;
  const int64_t rows = static_cast<int64_t>(a.M) * a.q_heads;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kAttnWaves + wave_index();
  const int lane = threadIdx.x & 63, piece = lane & 15, g = lane >> 4;
  if (row >= rows) return;
  const int token = static_cast<int>(row / a.q_heads);
  const int b = sequence_of_wave(a.offsets, a.cache.n_seqs, token);
  if (b >= a.cache.n_seqs) return;
  const Span s = span_of(a.offsets, b, a.M);
  if (token < s.off || token >= s.end) return;
  const int64_t start = a.starts[b];
  const int length = static_cast<int>(max(int64_t{0}, min(start + s.end - s.off, static_cast<int64_t>(a.cache.max_tokens))));
  int from, to;
  bounds_of(a, start, length, token - s.off, from, to);
  float v[E], l = 0.0f;
#pragma unroll
  for (int e = 0; e < E; ++e) v[e] = 0.0f;
  if (from < to) {
    // the parts begin where the row's tile does
    const int group = a.q_heads / a.cache.kv_heads, rows_of = static_cast<int64_t>(s.end - s.off) * group > many ? many_rows : few_rows;
    const int r = (token - s.off) * group + static_cast<int>(row % a.q_heads) % group;
    int base, unused;
    bounds_of(a, start, length, r / rows_of * rows_of / group, base, unused);
    base = base / kUnit * kUnit;
    const int p0 = min((from - base) / a.chunk, a.splits - 1), n = min((to - 1 - base) / a.chunk, a.splits - 1) - p0 + 1;
    const float2* heads = reinterpret_cast<const float2*>(a.part + a.splits * rows * D) + p0 * rows + row;
    const float* sums = a.part + (p0 * rows + row) * D + piece * E;
    const float2 head = lane < n ? heads[lane * rows] : make_float2(kNoReference, 0.0f);
    // the sums of four parts, one for each 16 lanes, on their way before they are used
    float next[E];
    auto fetch = [&](int p) {
      const float* x = sums + min(p + g, n - 1) * rows * D;
#pragma unroll
      for (int e = 0; e < E; e += 4) {
        const float4 y = *reinterpret_cast<const float4*>(x + e);
        next[e] = y.x, next[e + 1] = y.y, next[e + 2] = y.z, next[e + 3] = y.w;
      }
    };
    fetch(0);
    float m = head.x;
    m = fmaxf(m, lane_xor<1>(m));
    m = fmaxf(m, lane_xor<2>(m));
    m = fmaxf(m, lane_xor<4>(m));
    m = fmaxf(m, lane_xor<8>(m));
    m = column_max(m);
    const float f = __builtin_amdgcn_exp2f(head.x - m);
    l = head.y * f;
    l += lane_xor<1>(l);
    l += lane_xor<2>(l);
    l += lane_xor<4>(l);
    l += lane_xor<8>(l);
    l = column_sum(l);
    for (int p = 0; p < n; p += 4) {
      float x[E];
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = next[e];
      if (p + 4 < n) fetch(p + 4);
      const float w = __shfl(f, min(p + g, n - 1));
      // a part behind the last is not multiplied: what was read for it may be NaN
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = p + g < n ? __builtin_fmaf(x[e], w, v[e]) : v[e];
    }
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = column_sum(v[e]);
  }
  if (g == 0) finish<D, In>(v, l, piece, static_cast<In*>(a.out) + row * D);
}

// Which widths have the way by operands.  256 wide heads are better off without: there are
// no registers for more than a column tile a wave (a prompt of 4608, 16 heads on 4, bf16: 346
// us, 316 by the kernel for few).  So are 128 wide ones of fp16, whose two terms of queries and
// weights spill (32 heads on 8: 2000 rows behind 8000 tokens 217 us, 151 by the other; 8000 alone
// 135 and 88, behind 8000 651 and 518; four of 2400 to 1500 behind 7000 490 and 297).
constexpr bool by_operands(int head_dim, bool f16) { return head_dim == 64 || (head_dim == 128 && !f16); }
// Rows (tokens times query heads a key head) above which a sequence goes that way, which
// pays where many rows read the same keys.  One sequence: by what its tiles read in all (32
// heads of 128 on 8, bf16: 1000 rows behind 16000 tokens 111 us, 123 by the other; 4000 alone
// 62 and 31, behind 8000 198 and 246).  Of more only the mean is known here, and the two kernels
// run one after the other, so that a batch should go by one of them: by this one if the
// mean is long and the tiles are more than the CUs, as their lengths differ (24 heads of 64,
// fp16: 1001, 834 and 667 rows, 288 tiles, 450 us, 519 by the other; 32 heads of 128 on 8, bf16:
// four of 4000 to 2500 rows, 440 tiles, 81 and 87, of 2400 to 1500, 280 tiles, 276 and 255, of
// 1000 to 625, 128 tiles, 325 and 248), else by the other but for prompts that are much
// longer than the rest.
constexpr int kNever = 0x7fffffff;
int few_rows(int64_t n_seqs, int64_t rows, int64_t tiles, int64_t max_tokens) {
  if (n_seqs == 1) return rows > 896 && rows * max_tokens >= int64_t{1} << 23 ? 896 : kNever;
  if (rows / n_seqs <= 768) return 2048;
  return tiles > 256 ? 256 : kNever;
}
// Rows of a tile of the kernel for few: 16 where that is most sequences' number, else 32,
// which share what a unit costs (128 wide: with 8 rows of each of 16 sequences behind 4000
// tokens 20.4 us and 25.5, with 30 31.8 and 29.7, with 150 80.6 and 78.5; 64 wide: with 30
// 34.7 and 41.7, with 150 79 and 74).  Sums of 256 wide heads leave no registers for 32 (30
// rows: 31 us, 48 with 32; 150: 78 and 111), nor do 64 wide ones in fp16, whose weights are
// two terms (150: 103 with 32).
constexpr bool small_tiles(int head_dim, bool f16) { return head_dim == 256 || (head_dim == 64 && f16); }
constexpr int few_tile(int head_dim, bool f16, int64_t mean) {
  return small_tiles(head_dim, f16) || mean <= (head_dim == 64 ? 32 : 16) ? 16 : 32;
}
// Column tiles of a wave of the kernel for many rows: two are what its registers hold of
// 128 wide heads (256, and 28 bytes of scratch beside the loop), and of 64 wide ones four
// spilled (685 us where two took 359).
constexpr int kWideTiles = 2;
// A workgroup of four waves has 64 KB of LDS at D = 64 and a CU two of them, out of step:
// better where tiles are uneven and a wave's work on a unit is long (440 us against 514 with
// eight for three pieces behind 16000 tokens, 188 against 215 for a prompt of 4608, 143 against
// 168 in bf16).  128 wide heads have half the columns for as many bytes and are held back by the
// fetches of the units, which eight waves share (four pieces of 1000 tokens behind 8000 400 us
// against 436, of 600 behind 7000 277 against 249, a prompt of 4608 as fast).
constexpr int wide_waves(int head_dim) { return head_dim == 128 ? 8 : 4; }
constexpr int kWidest = 8;              // waves a CU
constexpr int64_t kMostOperands = int64_t{8} << 30;             // bytes
constexpr int64_t kMostSlots = 65535;   // the third side of a grid

int64_t tiles_bound(int64_t M, int64_t group, int64_t n_seqs, int64_t rows) {
  // one for every sequence that has rows, and one for every full tile
  return std::min(M * group / rows + std::min(n_seqs, M), M * ((group + rows - 1) / rows));
}

template <typename Kernel>
hipError_t launch_tiles(Kernel kernel, const Attention& a, int rows, int waves, int few, int many, hipStream_t stream) {
  const int64_t tiles = tiles_bound(a.M, a.q_heads / a.cache.kv_heads, a.cache.n_seqs, rows);
  const int64_t grid = tiles * a.cache.kv_heads;
  if (grid * 64 * waves >= (int64_t{1} << 32)) return hipErrorInvalidConfiguration;
  kernel<<<dim3(static_cast<unsigned>(grid), static_cast<unsigned>(a.splits)), dim3(64 * waves), 0, stream>>>(a, few, many);
  return hipGetLastError();
}

template <int D, typename In>
hipError_t launch_heads(const Attention& a, hipStream_t stream) {
  constexpr int kAll = 0x7fffffff;
  const int64_t rows = static_cast<int64_t>(a.M) * (a.q_heads / a.cache.kv_heads);
  hipError_t e = hipSuccess;
  constexpr bool kF16 = std::is_same_v<In, _Float16>;
  const int tile = few_tile(D, kF16, rows / a.cache.n_seqs);
  const int many = a.slots > 0 ? a.limit : kAll, few = a.cache.n_seqs > 1 ? a.limit : 0;
  if (a.slots == 0 || a.cache.n_seqs > 1) {
    if constexpr (small_tiles(D, kF16)) e = launch_tiles(attend_few<D, 1, In>, a, 16, kAttnWaves, 0, many, stream);
    else e = tile == 16 ? launch_tiles(attend_few<D, 1, In>, a, 16, kAttnWaves, 0, many, stream)
                        : launch_tiles(attend_few<D, 2, In>, a, 32, kAttnWaves, 0, many, stream);
  }
  int many_tile = tile;
  if constexpr (by_operands(D, kF16)) {
    constexpr int kWaves = wide_waves(D);
    many_tile = 16 * kWideTiles * kWaves;
    if (a.slots > 0 && e == hipSuccess) {
      const int64_t units = (a.cache.max_tokens + kUnit - 1) / kUnit;
      make_operands<D><<<dim3(static_cast<unsigned>((units + kAttnWaves - 1) / kAttnWaves),
                              static_cast<unsigned>(a.cache.kv_heads), static_cast<unsigned>(a.slots)),
                         dim3(kAttnThreads), 0, stream>>>(a, few);
      e = hipGetLastError();
    }
    if (a.slots > 0 && e == hipSuccess)
      e = launch_tiles(attend_many<D, kWideTiles, kWaves, In>, a, many_tile, kWaves, few, kAll, stream);
  }
  if (e != hipSuccess || a.splits == 1) return e;
  const int64_t out_rows = static_cast<int64_t>(a.M) * a.q_heads;
  const int64_t grid = (out_rows + kAttnWaves - 1) / kAttnWaves;
  if (grid * kAttnThreads >= (int64_t{1} << 32)) return hipErrorInvalidConfiguration;
  join_kernel<D, In><<<dim3(static_cast<unsigned>(grid)), dim3(kAttnThreads), 0, stream>>>(a, tile, a.slots == 0 ? kAll : few, many_tile);
  return hipGetLastError();
}

template <typename In>
hipError_t launch_type(const Attention& a, hipStream_t stream) {
  if (a.cache.head_dim == 64) return launch_heads<64, In>(a, stream);
  if (a.cache.head_dim == 128) return launch_heads<128, In>(a, stream);
  return launch_heads<256, In>(a, stream);
}

}  // namespace

AttentionPlan plan_cache_attention(int64_t M, int64_t q_heads, int64_t kv_heads, int head_dim, int64_t n_seqs,
                                   int64_t max_tokens, int64_t window, bool f16) {
  const int64_t group = q_heads / kv_heads, rows = M * group;
  AttentionPlan p;
  const int64_t wide_tile = 16 * kWidest * kWideTiles;
  const int limit = few_rows(n_seqs, rows, tiles_bound(M, group, n_seqs, wide_tile) * kv_heads, max_tokens);
  // long prompts: as many as there can be
  const int64_t unit_bytes_ = static_cast<int64_t>(head_dim / 8) * 1024 + 16 + 64;
  p.limit = limit;
  p.slot_units = (max_tokens + kUnit - 1) / kUnit + 4;          // and spare ones
  p.slots = n_seqs == 1 ? (rows > limit ? 1 : 0) : std::min(n_seqs, rows / (int64_t{1} + limit));
  // all of them or none: what has no slot there would have no kernel
  if (!by_operands(head_dim, f16) || p.slots > kMostSlots || p.slots * kv_heads * p.slot_units > kMostOperands / unit_bytes_)
    p.slots = 0;
  const size_t operands = static_cast<size_t>(p.slots) * kv_heads * p.slot_units * unit_bytes_;
  const bool wide = p.slots > 0;
  const int64_t tile = wide ? wide_tile : few_tile(head_dim, f16, rows / n_seqs);
  const int64_t work = std::max<int64_t>(1, tiles_bound(M, group, n_seqs, tile) * kv_heads);
  // Workgroups: few rows 1536, six a CU, which has room for three or four and finds many of
  // them short (64 chats of up to 8192 tokens, 8 key heads of 128: 70 us; 1024 72, 2048 76,
  // 512 86; 32 of up to 8000, 16 of 64: 45, 1024 53; 8 of up to 32000: 49, 1024 49, 768 54),
  // and no part under 1024 keys, eight units a wave, since joining parts costs a launch (16
  // chats that see 1024: one part 20 us, of 512 keys 23, of 256 21; one chat of 1000 tokens
  // 11 and 14).  Prompts a CU's full of rows for every CU.
  const int64_t wanted = wide ? 256 : 1536;
  const int64_t least = wide ? 16 * kUnit : 32 * kUnit;         // keys of a part
  const int64_t most = std::min<int64_t>((wanted + work - 1) / work, 64);   // one a lane where they are joined
  // of all the keys, as the workspace is for a call with any window, and then of those a
  // tile sees: no more parts
  auto cut = [&](int64_t span, int64_t parts) {
    parts = std::max<int64_t>(1, std::min(parts, span / least));
    p.chunk = static_cast<int>(((span + parts - 1) / parts + least - 1) / least * least);
    p.splits = static_cast<int>((span + p.chunk - 1) / p.chunk);
  };
  cut(max_tokens, most);
  p.parts = p.splits == 1 ? 0 : (static_cast<size_t>(p.splits) * static_cast<size_t>(M * q_heads) * (head_dim + 2) * 4 + 255) / 256 * 256;
  p.workspace = p.parts + operands;
  const int64_t seen = window + (tile + group - 1) / group + kUnit;
  if (window != 0 && seen < max_tokens) cut(seen, p.splits);
  return p;
}

hipError_t launch_cache_attention(const Attention& a, bool f16, hipStream_t stream) {
  return f16 ? launch_type<_Float16>(a, stream) : launch_type<uint16_t>(a, stream);
}

}  // namespace convrot
