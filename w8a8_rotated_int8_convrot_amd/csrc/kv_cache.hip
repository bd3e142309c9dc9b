// kv_cache.hip -- tokens into the paged 4-bit cache and back, and whole pages
// from place to place (layout: cache.hpp).
//
// One key or value head of one token, a row x of D values:
//   in:   v = x H_D / sqrt(D)    s = bf16(fp32(max |v| / 7))    c = rne(v / s), in [-7, 7]
//   out:  x' = rnd(s c H_D / sqrt(D))
// The rotation is the layer's own, with the head as its group: it spreads a
// head's few large dims over all of them, and it is never taken back where the
// attention reads, since (q H) . (k H) = D q . k.  The codes are taken in 64 bits:
// the sums of 16-bit values are then exact (of bf16 where a row's values lie within
// 2^37 of each other, else to 2^-53 of the largest), so that a code depends on
// nothing but its row, and this card's 64-bit multiply-adds run at the rate of its
// 32-bit ones.  A row that holds infinities or NaN gets the scale NaN.
//
// Eight tokens at multiples of eight share the words of their value codes, so
// they are one wave's work: eight lanes a token, D / 8 dims a lane.  The wave that
// has the first new token of such an octet takes all of its new ones, and keeps
// the other tokens' bits of the words it writes.
//
// Bound by the vector unit where there are many tokens: six to eight stages of
// 64-bit sums, three of them across lanes, then scale, code and check, some 37
// instructions a value (10246 tokens of 16 heads of 64: append 26.4 us, 2.0 TB/s,
// vector unit 63 % busy; read, without the check, 17.2, 3.1 TB/s, 55 %).  A
// division instead of the reciprocal: 38.  Several heads a wave, with the octet
// found once: no faster (26), for more registers.  64 tokens of 8 heads: 6.1 and
// 4.9 us, a launch and a chain of latencies (offsets, table, rows).
#include "cache.hpp"

namespace convrot {
namespace {

constexpr int kWaves = 4;               // a workgroup

__device__ inline double lane_xor8(double v, int t) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  auto move = [&](uint32_t w) {
    const float f = __uint_as_float(w);
    return static_cast<uint64_t>(__float_as_uint(t == 1 ? lane_xor<1>(f) : t == 2 ? lane_xor<2>(f) : lane_xor<4>(f)));
  };
  return __builtin_bit_cast(double, move(static_cast<uint32_t>(b)) | (move(static_cast<uint32_t>(b >> 32)) << 32));
}
__device__ inline float lane_xor8(float v, int t) {
  return t == 1 ? lane_xor<1>(v) : t == 2 ? lane_xor<2>(v) : lane_xor<4>(v);
}

__device__ inline float fused(float a, float b, float c) { return __builtin_fmaf(a, b, c); }
__device__ inline double fused(double a, double b, double c) { return __builtin_fma(a, b, c); }

// H_D of a row of D = 8 E values, lane c of eight holding [E c, E c + E).
template <int E, typename T>
__device__ inline void rotate_head(T (&v)[E], int c) {
#pragma unroll
  for (int h = 1; h < E; h <<= 1) {
#pragma unroll
    for (int i = 0; i < E; ++i) {
      if ((i & h) == 0) {
        const T a = v[i], b = v[i + h];
        v[i] = a + b;
        v[i + h] = a - b;
      }
    }
  }
  // the upper lane of a pair keeps the difference: its own value enters negated
#pragma unroll
  for (int t = 1; t < 8; t <<= 1) {
    const T sign = (c & t) != 0 ? T(-1) : T(1);
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = fused(v[i], sign, lane_xor8(v[i], t));
  }
}

template <int D> struct HeadScale;      // 1 / sqrt(D) in 64 bits
template <> struct HeadScale<64> { static constexpr double value = 0.125; };
template <> struct HeadScale<128> { static constexpr double value = 0.08838834764831844055; };
template <> struct HeadScale<256> { static constexpr double value = 0.0625; };

// The E / 8 words of a row's codes in this lane, and the row's scale as bf16 bits.
template <int D, typename In, int E = D / 8>
__device__ inline void encode(const uint4 (&raw)[E / 8], int c, uint32_t (&w)[E / 8], uint32_t& scale) {
  double v[E];
#pragma unroll
  for (int j = 0; j < E / 8; ++j) {
    float f[8];
    widen8<In>(raw[j], f);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[8 * j + i] = static_cast<double>(f[i]);
  }
  rotate_head(v, c);
  double top = 0.0;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    v[i] *= HeadScale<D>::value;
    top = fmax(top, fabs(v[i]));
  }
  top = fmax(top, lane_xor8(top, 1));
  top = fmax(top, lane_xor8(top, 2));
  top = fmax(top, lane_xor8(top, 4));
  // one value that is not finite makes every sum of its row so (fmax passes over NaN)
  const bool finite = fabs(v[0]) < __builtin_inf();
  // top / 7, rounded once: by the nearest to 1 / 7 and the remainder, which is exact
  constexpr double kSeventh = 1.0 / 7.0;
  const double near = top * kSeventh;
  const auto s16 = static_cast<__bf16>(static_cast<float>(__builtin_fma(__builtin_fma(-7.0, near, top), kSeventh, near)));
  const float s = static_cast<float>(s16);
  scale = __builtin_bit_cast(uint16_t, s16);
  if (!finite || !(s < __builtin_inff())) scale = 0x7fc0u;
  const bool coded = finite && s > 0.0f && s < __builtin_inff();
  // the whole number nearest to v / s by a reciprocal of 24 bits (added to 1.5 * 2^52 it
  // stands in the low bits): right where the remainder, which is exact, is below half a
  // scale; one that is not, about a code in a million, makes the wave divide
  const double sd = static_cast<double>(s), inverse = static_cast<double>(__builtin_amdgcn_rcpf(s));
  constexpr double kWhole = 6755399441055744.0;
  double worst = 0.0;
#pragma unroll
  for (int j = 0; j < E / 8; ++j) {
    w[j] = 0x88888888u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const double at = __builtin_fma(v[8 * j + i], inverse, kWhole);
      worst = fmax(worst, fabs(__builtin_fma(kWhole - at, sd, v[8 * j + i])));
      w[j] += static_cast<uint32_t>(__builtin_bit_cast(uint64_t, at)) << (4 * i);
    }
  }
  if (__any(coded && !(worst < 0.5 * sd && s >= 0x1p-120f))) {
#pragma unroll
    for (int j = 0; j < E / 8; ++j) {
      w[j] = 0x88888888u;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const double q = coded ? fmin(fmax(rint(v[8 * j + i] / sd), -7.0), 7.0) : 0.0;
        w[j] += static_cast<uint32_t>(static_cast<int>(q)) << (4 * i);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < E / 8; ++j) w[j] = coded ? w[j] : 0x88888888u;
}

template <int D, typename In, int E = D / 8>
__device__ inline void decode(const uint32_t (&w)[E / 8], uint32_t scale, int c, uint4 (&raw)[E / 8]) {
  float v[E];
#pragma unroll
  for (int j = 0; j < E / 8; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) v[8 * j + i] = static_cast<float>(static_cast<int>((w[j] >> (4 * i)) & 15u) - 8);
  rotate_head(v, c);                    // whole numbers up to 2048
  // (v s) / sqrt(D), the first product exact.  It may pass the largest fp32 where the second does not:
  // scales from 1 on enter 2^-8 times as large, which they hold exactly
  const float s = __uint_as_float(scale << 16);
  const bool large = s >= 1.0f;
  const float by = large ? s * 0x1p-8f : s;
  const float root = static_cast<float>(HeadScale<D>::value) * (large ? 0x1p8f : 1.0f);
#pragma unroll
  for (int j = 0; j < E / 8; ++j) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = (v[8 * j + i] * by) * root;
    raw[j] = narrow8<In>(f);
  }
}

// Words of eight rows (lanes 8 r + c) turned round: nibble j of row r's word goes
// to nibble r of row j's, by three exchanges of the half that is not one's own.
__device__ inline uint32_t turn_nibbles(uint32_t w, int r) {
  constexpr uint32_t kKeep[3] = {0x0f0f0f0fu, 0x00ff00ffu, 0x0000ffffu};
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    const uint32_t m = kKeep[k];
    const uint32_t other = static_cast<uint32_t>(__shfl_xor(static_cast<int>(w), 8 << k));
    const int by = 4 << k;
    w = (r >> k & 1) != 0 ? (w & ~m) | ((other & ~m) >> by) : (w & m) | ((other & m) << by);
  }
  return w;
}

// Row pointers and the tokens they go to, as convrot_cache_append's and
// convrot_cache_read's arguments; ROWS rows a wave.
template <typename In> struct Rows {
  In *k, *v;
  int64_t k_stride, v_stride;
  int M;
  const int32_t *starts, *offsets;
};

// Calls octet(b, o, row0, off, end) for every octet of tokens whose first row is
// among this wave's `count` rows: o the octet's number in sequence b, row0 the row
// of its first token, which need not be one of the rows [off, end) of b.
template <typename In, typename F>
__device__ inline void for_octets(const Cache& cache, const Rows<In>& rows, int first, int count, F&& octet) {
  const int lane = threadIdx.x & 63;
  int b = -1, off = 0, end = 0;
  int64_t at = 0;
  const int row = first + lane;
  bool leads = false;
  if (first >= rows.M) return;
  const int b0 = sequence_of_wave(rows.offsets, cache.n_seqs, first);
  if (lane < count && row < rows.M) {
    b = b0;
    if (b < cache.n_seqs && rows.offsets[b + 1] <= row) b = sequence_of(rows.offsets, cache.n_seqs, row);
    if (b < cache.n_seqs) {
      const Span s = span_of(rows.offsets, b, rows.M);
      off = s.off;
      end = s.end;
      at = static_cast<int64_t>(rows.starts[b]) + row - off;
      leads = off <= row && row < end && ((at & 7) == 0 || row == off);
    }
  }
  uint64_t todo = __ballot(leads);
  while (todo != 0) {
    const int l = __builtin_ctzll(todo);
    todo &= todo - 1;
    const int lb = __builtin_amdgcn_readlane(b, l), loff = __builtin_amdgcn_readlane(off, l);
    const int lend = __builtin_amdgcn_readlane(end, l);
    const int64_t lat = (static_cast<int64_t>(__builtin_amdgcn_readlane(static_cast<int>(at >> 32), l)) << 32) |
                        static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(at), l));
    octet(lb, lat >> 3, static_cast<int64_t>(first) + l - (lat & 7), loff, lend);
  }
}

// The unit of head h that holds octet o of sequence b, or null where no page of
// the cache is named for it.
__device__ inline uint8_t* unit_of(const Cache& c, int b, int64_t o, int h) {
  if (o < 0 || o * 8 >= c.max_tokens) return nullptr;
  const int at = static_cast<int>(o) * 8;
  const int64_t page = c.table[b * c.table_stride + (at >> c.page_shift)];
  if (page < 0 || page >= c.n_pages) return nullptr;
  const int units = 1 << (c.page_shift - 5);
  return c.pages + page * c.page_bytes + static_cast<int64_t>(h * units + ((at >> 5) & (units - 1))) * unit_bytes(c.head_dim);
}

template <int D, typename In>
__global__ __launch_bounds__(kWaves * 64) void append_kernel(Cache cache, Rows<const In> rows, int count) {
  constexpr int E = D / 8;
  const int lane = threadIdx.x & 63, r = lane >> 3, c = lane & 7, h = blockIdx.y;
  const int first = (static_cast<int>(blockIdx.x) * kWaves + static_cast<int>(threadIdx.x >> 6)) * count;
  for_octets(cache, rows, first, count, [&](int b, int64_t o, int64_t row0, int off, int end) {
    uint8_t* unit = unit_of(cache, b, o, h);
    if (unit == nullptr) return;
    const int64_t row = row0 + r;
    const bool live = row >= off && row < end;
    uint4 kr[E / 8], vr[E / 8];
    if (live) {
      const In* kp = rows.k + row * rows.k_stride + h * D + c * E;
      const In* vp = rows.v + row * rows.v_stride + h * D + c * E;
#pragma unroll
      for (int j = 0; j < E / 8; ++j) {
        kr[j] = reinterpret_cast<const uint4*>(kp)[j];
        vr[j] = reinterpret_cast<const uint4*>(vp)[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < E / 8; ++j) kr[j] = vr[j] = make_uint4(0, 0, 0, 0);
    }
    const int token = static_cast<int>(o & 3) * 8 + r;
    uint32_t w[E / 8], scale;
    encode<D, In>(kr, c, w, scale);
    if (live) {
      uint32_t* to = reinterpret_cast<uint32_t*>(unit + token * (D / 2) + c * (E / 2));
#pragma unroll
      for (int j = 0; j < E / 8; ++j) to[j] = w[j];
      if (c == 0) reinterpret_cast<uint16_t*>(unit + key_scales_at(D))[token] = static_cast<uint16_t>(scale);
    }
    encode<D, In>(vr, c, w, scale);
    if (live && c == 0) reinterpret_cast<uint16_t*>(unit + value_scales_at(D))[token] = static_cast<uint16_t>(scale);
    // the bits of the new tokens in a word
    const uint64_t lives = __ballot(live);
    uint32_t mine = 0;
#pragma unroll
    for (int t = 0; t < 8; ++t) mine |= (lives >> (8 * t) & 1) != 0 ? 15u << (4 * t) : 0u;
    uint32_t* words = reinterpret_cast<uint32_t*>(unit + value_codes_at(D)) + static_cast<int>(o & 3) * D + c * E + r;
#pragma unroll
    for (int j = 0; j < E / 8; ++j) {
      const uint32_t t = turn_nibbles(w[j], r);
      words[8 * j] = mine == ~0u ? t : (words[8 * j] & ~mine) | (t & mine);
    }
  });
}

template <int D, typename In>
__global__ __launch_bounds__(kWaves * 64) void read_kernel(Cache cache, Rows<In> rows, int count) {
  constexpr int E = D / 8;
  const int lane = threadIdx.x & 63, r = lane >> 3, c = lane & 7, h = blockIdx.y;
  const int first = (static_cast<int>(blockIdx.x) * kWaves + static_cast<int>(threadIdx.x >> 6)) * count;
  for_octets(cache, rows, first, count, [&](int b, int64_t o, int64_t row0, int off, int end) {
    const uint8_t* unit = unit_of(cache, b, o, h);
    const int64_t row = row0 + r;
    const bool live = row >= off && row < end;
    const int token = static_cast<int>(o & 3) * 8 + r;
    uint32_t kw[E / 8], vw[E / 8], ks = 0, vs = 0;
#pragma unroll
    for (int j = 0; j < E / 8; ++j) kw[j] = vw[j] = 0;
    if (unit != nullptr) {
      const uint32_t* from = reinterpret_cast<const uint32_t*>(unit + token * (D / 2) + c * (E / 2));
      const uint32_t* words =
          reinterpret_cast<const uint32_t*>(unit + value_codes_at(D)) + static_cast<int>(o & 3) * D + c * E + r;
#pragma unroll
      for (int j = 0; j < E / 8; ++j) {
        kw[j] = from[j];
        vw[j] = words[8 * j];
      }
      ks = reinterpret_cast<const uint16_t*>(unit + key_scales_at(D))[token];
      vs = reinterpret_cast<const uint16_t*>(unit + value_scales_at(D))[token];
    }
#pragma unroll
    for (int j = 0; j < E / 8; ++j) vw[j] = turn_nibbles(vw[j], r);
    uint4 out[E / 8];
    auto store = [&](In* to) {
#pragma unroll
      for (int j = 0; j < E / 8; ++j) reinterpret_cast<uint4*>(to)[j] = out[j];
    };
    if (rows.k != nullptr) {
      decode<D, In>(kw, ks, c, out);
      if (live) store(rows.k + row * rows.k_stride + h * D + c * E);
    }
    if (rows.v != nullptr) {
      decode<D, In>(vw, vs, c, out);
      if (live) store(rows.v + row * rows.v_stride + h * D + c * E);
    }
  });
}

// Rows a wave: the octets of long runs begin every eight rows, so that eight rows are one
// or two octets' work (append and read of 10246 tokens of 16 heads 43 us, 91 with a wave
// for each row); where a sequence brings few, each row begins an octet of its own, or most
// waves end at once, and a wave's octets would follow one another (64 sequences of one
// row 18 us, 43 with eight rows a wave; of up to eight 16.7 and 24.5; 512 of up to eight
// 44.9 and 44.6).
int rows_a_wave(int64_t M, int n_seqs) { return M >= int64_t{16} * n_seqs ? 8 : 1; }

template <typename Launch>
hipError_t by_rows(const Cache& c, int64_t M, Launch&& launch) {
  const int count = rows_a_wave(M, c.n_seqs);
  const int64_t grid = (M + kWaves * count - 1) / (kWaves * count);
  if (grid * kWaves * 64 >= (int64_t{1} << 32) || grid > 0x7fffffff) return hipErrorInvalidConfiguration;
  launch(dim3(static_cast<unsigned>(grid), static_cast<unsigned>(c.kv_heads)), count);
  return hipGetLastError();
}

// ---------------------------------------------------------------- pages

constexpr int kPairsALaunch = 256;      // 2 KB of the launch's arguments, which need no copy before it
constexpr int kCopyThreads = 256;
constexpr int kCopyLoads = 4;           // 16-byte pieces of a thread: at the copy rate (200 pages
                                        // of 68 KB in 32 layers: 165 us, 5.3 TB/s)
struct Pairs {
  int32_t src[kPairsALaunch], dst[kPairsALaunch];
};

__global__ __launch_bounds__(kCopyThreads) void copy_kernel(uint8_t* pages, int64_t layer_bytes, int64_t page_bytes, Pairs pairs) {
  const int64_t pieces = page_bytes / 16;
  uint8_t* layer = pages + blockIdx.z * layer_bytes;
  const auto* from = reinterpret_cast<const uint4*>(layer + pairs.src[blockIdx.y] * page_bytes);
  auto* to = reinterpret_cast<uint4*>(layer + pairs.dst[blockIdx.y] * page_bytes);
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kCopyThreads * kCopyLoads);
  from += first + threadIdx.x;
  to += first + threadIdx.x;
  if (first + kCopyThreads * kCopyLoads <= pieces) {
    const uint4 v0 = from[0], v1 = from[kCopyThreads], v2 = from[2 * kCopyThreads], v3 = from[3 * kCopyThreads];
    to[0] = v0, to[kCopyThreads] = v1, to[2 * kCopyThreads] = v2, to[3 * kCopyThreads] = v3;
  } else {
    for (int64_t i = first + threadIdx.x; i < pieces; i += kCopyThreads, from += kCopyThreads, to += kCopyThreads) *to = *from;
  }
}

}  // namespace

hipError_t launch_cache_append(const Cache& c, const void* k, int64_t k_stride, const void* v, int64_t v_stride, bool f16,
                               int64_t M, const int32_t* starts, const int32_t* offsets, hipStream_t stream) {
  return by_rows(c, M, [&](dim3 grid, int count) {
    auto go = [&](auto kernel, auto type) {
      using In = decltype(type);
      kernel<<<grid, dim3(kWaves * 64), 0, stream>>>(
          c, Rows<const In>{static_cast<const In*>(k), static_cast<const In*>(v), k_stride, v_stride, static_cast<int>(M),
                            starts, offsets},
          count);
    };
    if (f16) {
      if (c.head_dim == 64) go(append_kernel<64, _Float16>, _Float16{});
      else if (c.head_dim == 128) go(append_kernel<128, _Float16>, _Float16{});
      else go(append_kernel<256, _Float16>, _Float16{});
    } else {
      if (c.head_dim == 64) go(append_kernel<64, uint16_t>, uint16_t{});
      else if (c.head_dim == 128) go(append_kernel<128, uint16_t>, uint16_t{});
      else go(append_kernel<256, uint16_t>, uint16_t{});
    }
  });
}

hipError_t launch_cache_read(const Cache& c, void* k, int64_t k_stride, void* v, int64_t v_stride, bool f16, int64_t M,
                             const int32_t* starts, const int32_t* offsets, hipStream_t stream) {
  return by_rows(c, M, [&](dim3 grid, int count) {
    auto go = [&](auto kernel, auto type) {
      using In = decltype(type);
      kernel<<<grid, dim3(kWaves * 64), 0, stream>>>(
          c, Rows<In>{static_cast<In*>(k), static_cast<In*>(v), k_stride, v_stride, static_cast<int>(M), starts, offsets},
          count);
    };
    if (f16) {
      if (c.head_dim == 64) go(read_kernel<64, _Float16>, _Float16{});
      else if (c.head_dim == 128) go(read_kernel<128, _Float16>, _Float16{});
      else go(read_kernel<256, _Float16>, _Float16{});
    } else {
      if (c.head_dim == 64) go(read_kernel<64, uint16_t>, uint16_t{});
      else if (c.head_dim == 128) go(read_kernel<128, uint16_t>, uint16_t{});
      else go(read_kernel<256, uint16_t>, uint16_t{});
    }
  });
}

hipError_t launch_cache_copy(uint8_t* pages, int64_t layers, int64_t layer_bytes, int64_t page_bytes, const int32_t* src,
                             const int32_t* dst, int64_t n, hipStream_t stream) {
  constexpr int64_t kPiece = int64_t{kCopyThreads} * kCopyLoads * 16;
  const dim3 block(kCopyThreads);
  const auto pieces = static_cast<unsigned>((page_bytes + kPiece - 1) / kPiece);
  for (int64_t i0 = 0; i0 < n; i0 += kPairsALaunch) {
    Pairs p{};
    const int64_t here = n - i0 < kPairsALaunch ? n - i0 : kPairsALaunch;
    for (int64_t i = 0; i < here; ++i) {
      p.src[i] = src[i0 + i];
      p.dst[i] = dst[i0 + i];
    }
    copy_kernel<<<dim3(pieces, static_cast<unsigned>(here), static_cast<unsigned>(layers)), block, 0, stream>>>(
        pages, layer_bytes, page_bytes, p);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace convrot
