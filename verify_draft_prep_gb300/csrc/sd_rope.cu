// sd_rope.cu -- rotary positions of queries and keys (sd_rope) and the table of turns that they are
// made with (sd_rope_table).
//
// Pair i of a head, (a, b), at position p turns by the angle 2 pi p f_i:
//   a' = s (a cos - b sin),  b' = s (b cos + a sin).
// f_i is held as a 64-bit fraction of a turn, so that p f_i modulo a whole turn is one integer
// product: exact for every 32-bit position (an fp32 angle is off by 2^-7 radians at 10^5, and fp64
// arithmetic is slow here). The upper 32 bits, as a signed count of 2^-31 half turns, become fp32 and
// go to sincospif: the angle is off by 10^-7 radians at most, wherever the token stands.

#include <cmath>

#include "sd_kv.cuh"

namespace sdk {

struct RopeParams {
  const int32_t* pos;
  const uint64_t* turns;
  int n, D, rot, chunk, per_head;  // tokens of a CTA; units of a head
  int heads[2];
  float scale, sign;
  const uint16_t* x[2];
  uint16_t* y[2];
  long ld_x[2], hs_x[2], ld_y[2], hs_y[2];
};

constexpr int kRopeThreads = 256, kRopeAhead = 4;

template <int W>
struct RopeVec;
template <>
struct RopeVec<8> { using T = uint4; };
template <>
struct RopeVec<4> { using T = uint2; };
template <>
struct RopeVec<2> { using T = uint32_t; };
template <>
struct RopeVec<1> { using T = uint16_t; };

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

template <int W>
__device__ __forceinline__ void unpack(const typename RopeVec<W>::T& v, float (&f)[W]) {
  if constexpr (W == 1) {
    f[0] = bf16_bits_to_float(v);
  } else {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&v);
#pragma unroll
    for (int i = 0; i < W / 2; ++i) {
      f[2 * i] = bf16_lo(w[i]);
      f[2 * i + 1] = bf16_hi(w[i]);
    }
  }
}

template <int W>
__device__ __forceinline__ typename RopeVec<W>::T pack(const float (&f)[W]) {
  typename RopeVec<W>::T v;
  if constexpr (W == 1) {
    v = (uint16_t)pack_bf16(f[0], 0.f);
  } else {
    uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int i = 0; i < W / 2; ++i) w[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
  }
  return v;
}

// A CTA takes `chunk` tokens with all their heads: the cosines and sines are made once for each token
// and pair, into shared memory. A unit is W values of a head (HALVES: W of either half). A group of
// per_head threads has one unit each of the same head and goes over neighbouring heads, so that its
// factors stay in registers until the token ends. 2 bytes are read and 2 written for each value, and
// nothing else is large: bound by memory. 16384 tokens of 40 heads of 128: 60 us, 82% of the copy rate;
// half of each head turned, neighbours paired, 8192 tokens: 31 us, 80%; a step's 384 tokens of 72 heads
// of 64: 3.9 us in a graph, a launch and three dependent latencies.
template <int W, bool HALVES>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams P) {
  using T = typename RopeVec<W>::T;
  constexpr int kPairs = HALVES ? W : W / 2;  // of a unit
  extern __shared__ float2 s_cs[];            // [tokens][rot / 2]
  const int tid = threadIdx.x, half = P.rot / 2;
  const int tok0 = blockIdx.x * P.chunk, toks = min(P.chunk, P.n - tok0);
  for (int i = tid; i < toks * half; i += kRopeThreads) {
    const int t = i / half, p = i - t * half;
    const uint64_t turn = (uint64_t)(int64_t)P.pos[tok0 + t] * P.turns[p];
    float s, c;
    sincospif((float)(int32_t)(turn >> 32) * 4.656612873077393e-10f, &s, &c);
    s_cs[i] = make_float2(c * P.scale, s * P.scale * P.sign);
  }
  __syncthreads();

  const int groups = kRopeThreads / P.per_head, g = tid / P.per_head;
  const int e0 = tid - g * P.per_head;
  if (P.per_head <= kRopeThreads && g >= groups) return;
  const int all = P.heads[0] + P.heads[1], items = toks * all;
  const int turned = HALVES ? half / W : P.rot / W;  // units that turn; the others are copied
  // (heads of more units than threads: each thread takes several)
  for (int e = e0; e < P.per_head; e += kRopeThreads) {
    const int ng = groups > 0 ? groups : 1, per = (items + ng - 1) / ng;
    const int first = min(items, g * per), last = min(items, first + per);
    const bool turn = e < turned;
    const int d = HALVES ? (turn ? e * W : P.rot + (e - turned) * W) : e * W;
    int t = first / all, h = first - t * all, have = -1;
    float2 cs[kPairs];
    for (int i = first; i < last; i += kRopeAhead) {
      T a[kRopeAhead], b[kRopeAhead];
      int tk[kRopeAhead], hd[kRopeAhead];
#pragma unroll
      for (int k = 0; k < kRopeAhead; ++k) {
        tk[k] = t;
        hd[k] = h;
        if (i + k < last) {
          const int side = h >= P.heads[0];
          const uint16_t* x = P.x[side] + (long)(tok0 + t) * P.ld_x[side] +
                              (long)(side ? h - P.heads[0] : h) * P.hs_x[side] + d;
          a[k] = *reinterpret_cast<const T*>(x);
          if (HALVES && turn) b[k] = *reinterpret_cast<const T*>(x + half);
        }
        if (++h == all) {
          h = 0;
          ++t;
        }
      }
#pragma unroll
      for (int k = 0; k < kRopeAhead; ++k) {
        if (i + k >= last) break;
        const int side = hd[k] >= P.heads[0];
        uint16_t* y = P.y[side] + (long)(tok0 + tk[k]) * P.ld_y[side] +
                      (long)(side ? hd[k] - P.heads[0] : hd[k]) * P.hs_y[side] + d;
        if (!turn) {
          if (P.y[side] != P.x[side]) *reinterpret_cast<T*>(y) = a[k];
          continue;
        }
        if (tk[k] != have) {
          have = tk[k];
#pragma unroll
          for (int j = 0; j < kPairs; ++j) cs[j] = s_cs[have * half + e * kPairs + j];
        }
        float f[W];
        unpack<W>(a[k], f);
        if constexpr (HALVES) {
          float o[W];
          unpack<W>(b[k], o);
#pragma unroll
          for (int j = 0; j < W; ++j) {
            const float u = f[j] * cs[j].x - o[j] * cs[j].y, v = o[j] * cs[j].x + f[j] * cs[j].y;
            f[j] = u;
            o[j] = v;
          }
          *reinterpret_cast<T*>(y + half) = pack<W>(o);
        } else {
#pragma unroll
          for (int j = 0; j < kPairs; ++j) {
            const float u = f[2 * j] * cs[j].x - f[2 * j + 1] * cs[j].y;
            f[2 * j + 1] = f[2 * j + 1] * cs[j].x + f[2 * j] * cs[j].y;
            f[2 * j] = u;
          }
        }
        *reinterpret_cast<T*>(y) = pack<W>(f);
      }
    }
  }
}

template <int W, bool HALVES>
static int launch_rope(RopeParams& P, cudaStream_t stream) {
  P.per_head = HALVES ? P.rot / 2 / W + (P.D - P.rot) / W : P.D / W;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((P.n + P.chunk - 1) / P.chunk), 1, 1);
  cfg.blockDim = dim3(kRopeThreads, 1, 1);
  cfg.dynamicSmemBytes = (size_t)P.chunk * (P.rot / 2) * sizeof(float2);
  cfg.stream = stream;
  return cudaLaunchKernelEx(&cfg, rope_kernel<W, HALVES>, P) == cudaSuccess ? SD_OK : SD_E_LAUNCH;
}

}  // namespace sdk

extern "C" int sd_rope_launch(int n, int Hq, int Hk, int D, int rot, int pairs,
                              const int32_t* positions, const uint64_t* turns, float scale,
                              int inverse, const void* q, long ld_q, long hs_q, void* q_out,
                              long ld_qo, long hs_qo, const void* k, long ld_k, long hs_k,
                              void* k_out, long ld_ko, long hs_ko, cudaStream_t stream) {
  sdk::RopeParams P;
  P.pos = positions;
  P.turns = turns;
  P.n = n;
  P.D = D;
  P.rot = rot;
  P.heads[0] = Hq;
  P.heads[1] = Hk;
  P.scale = scale;
  P.sign = inverse ? -1.f : 1.f;
  P.x[0] = (const uint16_t*)q;
  P.x[1] = (const uint16_t*)k;
  P.y[0] = (uint16_t*)q_out;
  P.y[1] = (uint16_t*)k_out;
  P.ld_x[0] = ld_q;
  P.hs_x[0] = hs_q;
  P.ld_x[1] = ld_k;
  P.hs_x[1] = hs_k;
  P.ld_y[0] = ld_qo;
  P.hs_y[0] = hs_qo;
  P.ld_y[1] = ld_ko;
  P.hs_y[1] = hs_ko;
  // Tokens of a CTA: a step's few spread over the SMs, a prompt's share their CTA's setup. With 1, 2, 4,
  // 8, 16: 384 tokens 4.9, 3.9, 4.1, 5.3, 7.7 us, 8192 42.9, 36.0, 32.7, 31.7, 30.8, 16384 124.7, 84.1,
  // 68.9, 60.3, 60.0.
  int dev = 0;
  const int places = 2 * sdk::device_sms(dev);
  if (places == 0) return SD_E_DEVICE;
  P.chunk = n / places < 2 ? 2 : n / places > 16 ? 16 : n / places;
  // The widest accesses that every part of a head allows: 16 bytes, else 8 (halves) or a pair.
  if (pairs == SD_ROPE_HALVES) {
    if (rot % 16 == 0) return sdk::launch_rope<8, true>(P, stream);
    if (rot % 8 == 0) return sdk::launch_rope<4, true>(P, stream);
    return sdk::launch_rope<1, true>(P, stream);
  }
  return rot % 8 == 0 ? sdk::launch_rope<8, false>(P, stream)
                      : sdk::launch_rope<2, false>(P, stream);
}

// Host arithmetic in fp64: radians a position, then turns as a fraction of 2^64.
extern "C" void sd_rope_table_make(int rot, double base, int kind, double factor,
                                   double original_len, double low, double high, uint64_t* turns,
                                   float* scale) {
  const double pi = 3.14159265358979323846;
  double first = 0, last = 0;
  *scale = 1.f;
  if (kind == SD_ROPE_NTK) base *= std::pow(factor, rot / std::fmax(1.0, rot - 2.0));
  if (kind == SD_ROPE_YARN) {
    auto at = [&](double t) {
      return rot * std::log(original_len / (t * 2 * pi)) / (2 * std::log(base));
    };
    first = std::fmax(std::floor(at(high)), 0.0);
    last = std::fmin(std::ceil(at(low)), rot - 1.0);
    *scale = (float)(0.1 * std::log(factor) + 1.0);
  }
  for (int i = 0; i < rot / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rot), keep = 1;
    if (kind == SD_ROPE_LINEAR) keep = 0;
    if (kind == SD_ROPE_BANDS)
      keep = std::fmin(std::fmax((original_len * f / (2 * pi) - low) / (high - low), 0.0), 1.0);
    if (kind == SD_ROPE_YARN)
      keep = 1 - std::fmin(std::fmax((i - first) / std::fmax(last - first, 0.001), 0.0), 1.0);
    f = f * keep + f / factor * (1 - keep);
    const double t = std::fmod(f / (2 * pi), 1.0);
    turns[i] = (uint64_t)std::floor(std::ldexp(t, 64));
  }
}
