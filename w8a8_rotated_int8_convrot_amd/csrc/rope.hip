// rope.hip -- rotary positions on the heads of queries and keys.
//
// Pair (a, b) of a head at position p, with the pair's frequency f (radians a
// position) and a factor c:
//   phi = p f       a' = c (a cos phi - b sin phi)       b' = c (b cos phi + a sin phi)
// and the dims behind the turned part copied.  phi of a far position has more
// digits than fp32: p f / (2 pi) is taken in 64 bits, its whole turns are
// dropped there, and what is left, at most half a turn, goes to fp32 (2^-26
// turns, below the last digit of a sine), where the sine, the cosine and the
// products are.  One rounding to 16 bits at the end.
//
// Bound by memory: 4 bytes an element.  A workgroup takes a few tokens, makes
// their sines and cosines once in LDS for all heads, and then moves vectors of
// up to 16 bytes; a thread has up to three of them in flight (4608 tokens of 48
// heads of 128, half of each turned: 18.8 us, 6.0 TB/s; four 19.7, two 19.0).  An
// item behind the last is the last again, not stored: with the loads under a
// condition they went through scratch memory (29 us).  One token: 2.5 us, the
// launch.
#include "convrot_internal.hpp"
#include "rotate_device.hpp"

namespace convrot {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxTokens = 4;       // a workgroup
constexpr int kRopeInFlight = 3;        // vectors a thread has loaded at a time

// N 16-bit values as one memory access.
template <int N> struct Raw;
template <> struct Raw<1> { using type = uint16_t; };
template <> struct Raw<2> { using type = uint32_t; };
template <> struct Raw<4> { using type = uint32_t __attribute__((ext_vector_type(2))); };
template <> struct Raw<8> { using type = uint32_t __attribute__((ext_vector_type(4))); };

template <typename In, int N>
__device__ inline void widen(const typename Raw<N>::type& r, float (&v)[N]) {
  In e[N];
  __builtin_memcpy(e, &r, sizeof e);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (std::is_same_v<In, _Float16>) v[i] = static_cast<float>(e[i]);
    else v[i] = __uint_as_float(static_cast<uint32_t>(e[i]) << 16);
  }
}
template <typename In, int N>
__device__ inline typename Raw<N>::type narrow(const float (&v)[N]) {
  typename Raw<N>::type r;
  if constexpr (N == 1) {
    r = static_cast<uint16_t>(pack2<In>(v[0], 0.0f));
  } else {
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) w[i] = pack2<In>(v[2 * i], v[2 * i + 1]);
    __builtin_memcpy(&r, w, sizeof r);
  }
  return r;
}

// The dims behind the turned ones of so many heads, N values an item.
template <typename In, int N, typename Place>
__device__ inline void copy_rest(int heads, const Rope& p, int tid, Place&& place) {
  using R = typename Raw<N>::type;
  const int each = (p.head_dim - p.rot_dim) / N, items = heads * each;
  for (int i0 = tid; i0 < items; i0 += kRopeThreads * kRopeInFlight) {
    R v[kRopeInFlight];
    In* to[kRopeInFlight];
#pragma unroll
    for (int j = 0; j < kRopeInFlight; ++j) {
      int t, e;                         // behind the last item the last again, not stored
      const In* from;
      place(min(i0 + j * kRopeThreads, items - 1), each, t, e, from, to[j]);
      to[j] += p.rot_dim + N * e;
      v[j] = *reinterpret_cast<const R*>(from + p.rot_dim + N * e);
    }
#pragma unroll
    for (int j = 0; j < kRopeInFlight; ++j)
      if (i0 + j * kRopeThreads < items) *reinterpret_cast<R*>(to[j]) = v[j];
  }
}

// V pairs are one item: in the half layout two vectors of V values rot / 2
// apart, interleaved one vector of 2 V.
template <typename In, int V, bool INTERLEAVED>
__global__ __launch_bounds__(kRopeThreads) void rope_kernel(Rope p, int tokens) {
  extern __shared__ float2 turn[];      // [tokens][rot / 2]: cosine, sine
  const int tid = threadIdx.x;
  const int64_t m0 = static_cast<int64_t>(blockIdx.x) * tokens;
  const int here = static_cast<int>(min(static_cast<int64_t>(tokens), p.M - m0));
  const int half = p.rot_dim / 2;
  const int heads = static_cast<int>(p.part[0].heads + p.part[1].heads);

  // item i of so many a head: its token and place in the head, and the head's
  // first value in the input and the output
  const int first = static_cast<int>(p.part[0].heads);
  const auto* q_in = static_cast<const In*>(p.part[0].in) + m0 * p.part[0].in_stride;
  const auto* k_in = static_cast<const In*>(p.part[1].in) + m0 * p.part[1].in_stride;
  auto* q_out = static_cast<In*>(p.part[0].out) + m0 * p.part[0].out_stride;
  auto* k_out = static_cast<In*>(p.part[1].out) + m0 * p.part[1].out_stride;
  const int64_t q_in_stride = p.part[0].in_stride, k_in_stride = p.part[1].in_stride;
  const int64_t q_out_stride = p.part[0].out_stride, k_out_stride = p.part[1].out_stride;
  auto place = [&](int i, int per_head, int& t, int& e, const In*& from, In*& to) {
    const int th = static_cast<int>(static_cast<unsigned>(i) / static_cast<unsigned>(per_head));
    e = i - th * per_head;
    t = static_cast<int>(static_cast<unsigned>(th) / static_cast<unsigned>(heads));
    const int h = th - t * heads;
    const bool second = h >= first;
    const int at = (second ? h - first : h) * p.head_dim;
    from = (second ? k_in : q_in) + (t * (second ? k_in_stride : q_in_stride) + at);
    to = (second ? k_out : q_out) + (t * (second ? k_out_stride : q_out_stride) + at);
  };
  // what is not turned first: its loads are under way while the sines are made
  if (p.rot_dim != p.head_dim) {
    if (p.rot_dim % 8 == 0) copy_rest<In, 8>(here * heads, p, tid, place);
    else copy_rest<In, 2>(here * heads, p, tid, place);
  }
  for (int i = tid; i < here * half; i += kRopeThreads) {
    const int t = i / half;
    const double turns = static_cast<double>(p.positions[m0 + t]) * (p.freqs[i - t * half] * 0.15915494309189533577);
    const float left = static_cast<float>(turns - rint(turns));
    float s, c;
    sincospif(2.0f * left, &s, &c);
    turn[i] = make_float2(c * p.scale, (p.inverse ? -s : s) * p.scale);
  }
  __syncthreads();
  constexpr int kV = INTERLEAVED ? 2 * V : V;
  using R = typename Raw<kV>::type;
  const int turned = half / V;

  const int items = here * heads * turned;
  for (int i0 = tid; i0 < items; i0 += kRopeThreads * kRopeInFlight) {
    R a[kRopeInFlight], b[kRopeInFlight];
    In* to[kRopeInFlight];
    const float2* cs[kRopeInFlight];
#pragma unroll
    for (int j = 0; j < kRopeInFlight; ++j) {
      int t, e;
      const In* from;
      place(min(i0 + j * kRopeThreads, items - 1), turned, t, e, from, to[j]);
      to[j] += e * kV;
      cs[j] = turn + t * half + e * V;
      a[j] = *reinterpret_cast<const R*>(from + e * kV);
      if constexpr (!INTERLEAVED) b[j] = *reinterpret_cast<const R*>(from + e * kV + half);
    }
#pragma unroll
    for (int j = 0; j < kRopeInFlight; ++j) {
      if (i0 + j * kRopeThreads < items) {
        float x[kV], y[kV], u[kV], w[kV];
        widen<In, kV>(a[j], x);
        if constexpr (INTERLEAVED) {
#pragma unroll
          for (int v = 0; v < V; ++v) {
            const float2 f = cs[j][v];
            u[2 * v] = __builtin_fmaf(x[2 * v], f.x, -(x[2 * v + 1] * f.y));
            u[2 * v + 1] = __builtin_fmaf(x[2 * v + 1], f.x, x[2 * v] * f.y);
          }
        } else {
          widen<In, kV>(b[j], y);
#pragma unroll
          for (int v = 0; v < V; ++v) {
            const float2 f = cs[j][v];
            u[v] = __builtin_fmaf(x[v], f.x, -(y[v] * f.y));
            w[v] = __builtin_fmaf(y[v], f.x, x[v] * f.y);
          }
          *reinterpret_cast<R*>(to[j] + half) = narrow<In, kV>(w);
        }
        *reinterpret_cast<R*>(to[j]) = narrow<In, kV>(u);
      }
    }
  }
}

template <typename In, int V, bool INTERLEAVED>
hipError_t launch_width(const Rope& p, hipStream_t stream) {
  // the more tokens, the more of their vectors a thread has in flight, as long as
  // every CU still has two workgroups (4608 tokens: four a workgroup 18.9 us, two 19.2, one
  // 22.6)
  int tokens = 1;
  while (tokens < kRopeMaxTokens && p.M >= int64_t{4} * tokens * num_cus()) tokens *= 2;
  const int64_t grid = (p.M + tokens - 1) / tokens;
  if (grid * kRopeThreads >= (int64_t{1} << 32)) return hipErrorInvalidConfiguration;
  rope_kernel<In, V, INTERLEAVED><<<dim3(static_cast<unsigned>(grid)), dim3(kRopeThreads),
                                    static_cast<size_t>(tokens) * (p.rot_dim / 2) * sizeof(float2), stream>>>(p, tokens);
  return hipGetLastError();
}

// The widest vectors that a head's turned part divides into.
template <typename In>
hipError_t launch_type(const Rope& p, hipStream_t stream) {
  const int pairs = p.rot_dim / 2;
  if (p.interleaved) {
    if (pairs % 4 == 0) return launch_width<In, 4, true>(p, stream);
    return pairs % 2 == 0 ? launch_width<In, 2, true>(p, stream) : launch_width<In, 1, true>(p, stream);
  }
  if (pairs % 8 == 0) return launch_width<In, 8, false>(p, stream);
  if (pairs % 4 == 0) return launch_width<In, 4, false>(p, stream);
  return pairs % 2 == 0 ? launch_width<In, 2, false>(p, stream) : launch_width<In, 1, false>(p, stream);
}

}  // namespace

hipError_t launch_rope(const Rope& p, bool f16, hipStream_t stream) {
  return f16 ? launch_type<_Float16>(p, stream) : launch_type<uint16_t>(p, stream);
}

}  // namespace convrot
