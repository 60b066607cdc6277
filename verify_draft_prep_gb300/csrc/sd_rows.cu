// sd_rows.cu -- rows cut by top-k, top-p and min-p: as probability rows (sd_truncate), or one token
// drawn from each by a given random number (sd_sample).
//
// The entries of a row stand in order, larger first and equal ones by their index, and what is kept
// is always a prefix of that order: the shortest of three. With weights w (the probabilities, or
// exp((l - l_max) / T)) the first top_k entries, of those the ones before which less than top_p of
// their sum lies, and the ones with w >= min_p w_max. A draw is a place in the running sum too. So
// every question is one for a place in the order, by count or by sum, and the row is never sorted: a
// histogram over its values answers them.
//
// Logits are bf16: a row has at most 65536 different values, so a histogram of all of them holds the
// row exactly, and w is needed once for each value that occurs instead of once for each entry. That is
// what lets the sums be exact enough for whole numbers to come out right: w in pairs of fp32 (2^-43), and
// from there on whole numbers of 2^-62 of the largest weight (81 bits), products with top-p and the
// drawn number among them, so that nothing is rounded however many bins there are. Probabilities have 32
// bits: the histogram is over their upper 16, with the sums of the lower 16 in whole numbers, and the
// one bin in question is resolved by reading the row again (from L2).
//
// Two kernels. quick_kernel has 8192 bins, for logits of magnitude 2^-15 to 2^17 (and zero) and
// probabilities from 2^-63 on: 32 or 64 KB, so that four or two CTAs are on an SM at a time and one
// row's search hides behind another's reading. A row that needs more (a cut or a draw within values
// that have no bin of their own, rows of odd scales) is marked, and rows_kernel, whose histogram has a
// bin for every value, does the marked rows. A row is a CTA's work, or a cluster's where rows are few:
// each CTA counts its part, then each scans its share of the bins over all of the cluster's histograms
// through distributed shared memory, and one warp does the search.

#include "sd_kv.cuh"
#include "sd_tc.cuh"

namespace sdk {

constexpr int kRowThreads = 1024, kRowWarps = kRowThreads / 32;
constexpr int kHistBytes = 131072;
constexpr int kMostClusters = 8;
// Sums are multiples of 2^-62 of the largest weight (logits), of the power of two above it or of one
// (probabilities): with up to 2^19 entries they have up to 81 bits, three numbers of 27 for a warp's
// reduction. (As multiples of 2^-43 in 64 bits every bin was rounded by up to 2^-44, and thousands of
// bins made it 2^-36 of a sum. With four numbers, of 2^-63: one token of each of 1024 rows 347 us
// against 345.)
constexpr int kSumBits = 62;
constexpr double kSumUnit = 0x1p62;

struct RowsParams {
  const void* rows;
  long ld;
  int J, V, part, vec;  // entries of a CTA's part; whether rows allow 16-byte loads
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  float* probs;  // sd_truncate
  long ld_out;
  int vec_out;
  const float* u;  // sd_sample
  int32_t* tokens;
  float* prob;
  int32_t* kept;
  int32_t* err;
  int n_rows;
};

// What marks a row that quick_kernel leaves to rows_kernel, in its output.
constexpr int32_t kMarkToken = -2147483647 - 1;
constexpr float kMarkProb = -1.f;

typedef unsigned __int128 u128;

// A value's place: entries of larger values and their sum, how many entries have the value, and the
// weight of each (in units of the sums).
struct Border {
  uint32_t key, above, count;
  unsigned long long w;
  u128 sum;
};

struct RowShared {
  float2 two_to[64];               // 2^(j / 64) as pairs
  uint32_t warp_count[kRowWarps];
  u128 warp_sum[kRowWarps];
  uint32_t rank_count[kMostClusters];
  u128 rank_sum[kMostClusters];
  uint32_t rank_top[kMostClusters];
  uint32_t rank_eq[kMostClusters];
  Border found, inside;             // a bin, by the CTA that holds it; an entry of it, by each CTA
  uint32_t low[256];                // counts of the sub-bins
  unsigned long long low_sum[256];  // sums of what lies below them
  uint32_t merged[256];
  unsigned long long merged_sum[256];
  float2 per_unit;  // log2(e) / T as a pair
  int index;
};

// 2^n in fp64, n from -1000 to 1000.
__device__ __forceinline__ double two_to_the(int n) {
  return __longlong_as_double((long long)(1023 + n) << 52);
}
__device__ __forceinline__ FF ff_sum(float a, float b) { return ff_two_sum(a, b); }

// 2^y for y = d c (pairs), y <= 0, as a count of 2^-62 (0 below 2^-62): k / 64 is y's nearest multiple
// of 2^-6, 2^(k/64) from the table, and the rest e^u with |u| <= 0.0055, whose terms from the third on
// need only fp32.
__device__ __forceinline__ unsigned long long weight62(FF d, float2 c, const float2* two_to) {
  const float p = d.hi * c.x;
  const float e = fmaf(d.hi, c.x, -p) + fmaf(d.hi, c.y, d.lo * c.x);
  const int k = __float2int_rn(p * 64.f);
  const FF g = ff_sum(fmaf((float)k, -0.015625f, p), e);
  constexpr float kLn2Hi = 0.69314718055994531f;
  constexpr float kLn2Lo = (float)(0.69314718055994530942 - (double)0.69314718055994531f);
  const float uh = g.hi * kLn2Hi;
  const float ul = fmaf(g.hi, kLn2Hi, -uh) + fmaf(g.hi, kLn2Lo, g.lo * kLn2Hi);
  const float q = uh * uh;
  const float ql = fmaf(uh, uh, -q) + 2.f * uh * ul;
  const float cube = q * uh * fmaf(uh, fmaf(uh, 1.f / 120.f, 1.f / 24.f), 1.f / 6.f);
  const FF r = ff_sum(uh, 0.5f * q);
  const float rl = r.lo + (ul + fmaf(0.5f, ql, cube));
  const float2 t = two_to[k & 63];
  const float ph = t.x * r.hi;
  const float pl = fmaf(t.x, r.hi, -ph) + fmaf(t.x, rl, t.y * r.hi);
  const FF s = ff_sum(t.x, ph);
  const float lo = s.lo + pl + t.y;
  const float up = __uint_as_float((uint32_t)(127 + kSumBits + (k >> 6)) << 23);
  const long long w = (long long)__float2ull_rz(s.hi * up) + __float2ll_rn(lo * up);
  return p > (float)-kSumBits ? (unsigned long long)w : 0;
}

// The warp's sum by its integer reduction; the sum is below 2^81.
__device__ __forceinline__ u128 warp_sum(u128 v) {
  const uint32_t a = __reduce_add_sync(0xffffffffu, (uint32_t)v & 0x7ffffffu);
  const uint32_t b = __reduce_add_sync(0xffffffffu, (uint32_t)(v >> 27) & 0x7ffffffu);
  const uint32_t c = __reduce_add_sync(0xffffffffu, (uint32_t)(v >> 54));
  return (u128)(a + ((unsigned long long)b << 27)) + ((u128)c << 54);
}
__device__ __forceinline__ uint32_t from_lane(uint32_t v, int lane) {
  return __shfl_sync(0xffffffffu, v, lane);
}
__device__ __forceinline__ u128 from_lane(u128 v, int lane) {
  return (u128)__shfl_sync(0xffffffffu, (unsigned long long)(v >> 64), lane) << 64 |
         __shfl_sync(0xffffffffu, (unsigned long long)v, lane);
}
__device__ __forceinline__ uint32_t from_below(uint32_t v, int by) {
  return __shfl_up_sync(0xffffffffu, v, by);
}
__device__ __forceinline__ unsigned long long from_below(unsigned long long v, int by) {
  return __shfl_up_sync(0xffffffffu, v, by);
}
__device__ __forceinline__ u128 from_below(u128 v, int by) {
  return (u128)__shfl_up_sync(0xffffffffu, (unsigned long long)(v >> 64), by) << 64 |
         __shfl_up_sync(0xffffffffu, (unsigned long long)v, by);
}
template <typename T>
__device__ __forceinline__ T warp_before(T v) {  // the sum over the lanes before this one
  const int lane = threadIdx.x & 31;
  T x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = from_below(x, o);
    if (lane >= o) x += y;
  }
  return x - v;
}

__device__ __forceinline__ double sum_double(u128 v) {
  return fma((double)(unsigned long long)(v >> 64), 0x1p64, (double)(unsigned long long)v);
}
// x * sum for 0 <= x <= 1, exact but for the places below 1, which are cut (and said to be there).
__device__ __forceinline__ u128 share_of(float x, u128 sum, bool& more) {
  const uint32_t b = __float_as_uint(x);
  const int down = 150 - max(1, (int)(b >> 23));  // x is its 24-bit significand times 2^-down
  const u128 all = sum * ((b >> 23 ? 0x800000u : 0u) | (b & 0x7fffffu));
  more = down > 127 ? all != 0 : (all & (((u128)1 << down) - 1)) != 0;
  return down > 127 ? (u128)0 : all >> down;
}
// The places in a running sum of `total` that a draw (u) and a top-p ask for: where u * kept lies, and the
// last one before top_p * kept.
__device__ __forceinline__ u128 draw_place(float u, u128 kept, u128 total) {
  bool more;
  const u128 g = share_of(u > 0.f ? fminf(u, 1.f) : 0.f, kept, more);
  return g < total ? g : total - 1;
}
__device__ __forceinline__ u128 last_place(float top_p, u128 kept, u128 total) {
  bool more;
  const u128 g = share_of(fmaxf(top_p, 0.f), kept, more);
  return more ? (g < total ? g : total - 1) : g == 0 ? (u128)0 : g - 1;
}
// d / w in whole numbers, most + 1 <= 2^19 or less: a quotient of fp32, put right.
__device__ __forceinline__ uint32_t quotient(u128 d, unsigned long long w, uint32_t most) {
  w = max(w, 1ull);
  const float f = fmaf((float)(unsigned long long)(d >> 32), 0x1p32f, (float)(uint32_t)d);
  uint32_t q = (uint32_t)fminf(__fdividef(f, (float)w), (float)most);
  const u128 p = (u128)w * q;
  if (p > d) --q;
  else if (d - p >= w) ++q;
  return min(q, most);
}
// `units` < 2^44 of 2^by, to nearest.
__device__ __forceinline__ u128 shifted(unsigned long long units, int by) {
  if (by >= 0) return (u128)units << by;
  return by < -62 ? 0 : ((units >> (-by - 1)) + 1) >> 1;
}

// Orderable keys. Logits: 16 bits, ascending with the value, both zeros alike; 0 for what is never
// kept (-inf, NaN). Probabilities: their bits; 0 for what is not above 0, and 1 for what is above 1.
__device__ __forceinline__ uint32_t logit_key(uint32_t b) {
  if (b == 0x8000u) b = 0;
  const uint32_t k = b & 0x8000u ? ~b & 0xffffu : b | 0x8000u;
  return k <= 0x7fu || k > 0xff80u ? 0u : k;
}
__device__ __forceinline__ float logit_value(uint32_t k) {
  return __uint_as_float((k & 0x8000u ? k & 0x7fffu : ~k & 0xffffu) << 16);
}
// The least key whose logit weighs min_p (0 < min_p < 1) of the largest one, in fp64.
__device__ __forceinline__ uint32_t least_logit_key(float top_value, float T, float min_p) {
  const double t = (double)top_value + fmin(fmax((double)T, 0x1p-100), 0x1p100) * log((double)min_p);
  const uint32_t o = orderable(__double2float_ru(t));
  return o & 0x80000000u ? (o + 0xffffu) >> 16 : o >> 16;
}
// Weights, as counts of 2^-62, tell entries apart to 2^-43 down to this share of the largest; below it they
// have fewer places, and then none.
constexpr float kLeastShare = 0x1p-16f;
__device__ __forceinline__ uint32_t prob_key(uint32_t b) {
  return b - 1u < 0x7f800000u ? min(b, 0x3f800000u) : 0u;
}

// What a kept entry's probability is made with: 1 over the sum of those kept, a pair, for weights in units of
// the largest (logits) or as they are but for a power of two (probabilities). A probability is rounded
// once (2^-24). A logit's distance from the largest is rounded to fp32 (2^-24 of it, which is as much of
// the result for each nat), its exponential is fp32's (2^-22), and two products: 2048 rows of 201088
// logits take 975 us so, 997 with the distance as a pair.
struct KeptValue {
  float2 inv;
  float2 per_unit;
  float top_value, scale;

  template <bool PROBS>
  __device__ __forceinline__ float of(uint32_t key) const {
    if (PROBS) {
      const float x = __uint_as_float(key) * scale;
      return fmaf(x, inv.x, x * inv.y);
    }
    const float d = logit_value(key) - top_value;
    const float y = d * per_unit.x;
    // (the product's rounding error goes into a factor)
    const float r = fmaf(d, per_unit.x, -y) + d * per_unit.y;
    const float x = exp2f(y) * fmaf(r, 0.69314718f, 1.f);
    return y > -160.f ? fmaf(x, inv.x, x * inv.y) : 0.f;
  }
};
__device__ __forceinline__ float2 pair_of(double x) {
  const float hi = (float)x;
  return make_float2(hi, (float)(x - (double)hi));
}

template <bool PROBS>
struct RowReader {
  const RowsParams& P;
  const void* row;
  int begin, end;  // this CTA's entries

  __device__ __forceinline__ uint32_t key_at(int i) const {
    return PROBS ? prob_key(__ldg((const uint32_t*)row + i))
                 : logit_key(__ldg((const uint16_t*)row + i));
  }

  // f(words, n) for the part in any order: 16 bytes at a time, or one entry (n = 1, in the word's
  // lower half for logits).
  template <typename F>
  __device__ __forceinline__ void raw(int first, int step, F f) const {
    constexpr int N = PROBS ? 4 : 8;
    int i0 = begin + first;
    if (P.vec) {
      const int vecs = (end - begin) / N;
      const uint4* p = reinterpret_cast<const uint4*>((const char*)row + (size_t)begin * (PROBS ? 4 : 2));
      constexpr int kAhead = 4;  // loads in flight
      uint4 x[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (first + k * step < vecs) x[k] = __ldg(p + first + k * step);
      for (int v = first; v < vecs; v += kAhead * step) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const int at = v + k * step;
          if (at >= vecs) break;
          const uint32_t now[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
          if (at + kAhead * step < vecs) x[k] = __ldg(p + at + kAhead * step);
          f(now, N);
        }
      }
      i0 += vecs * N;
    }
    for (int i = i0; i < end; i += step) {
      const uint32_t now[4] = {
          PROBS ? __ldg((const uint32_t*)row + i) : (uint32_t)__ldg((const uint16_t*)row + i), 0, 0, 0};
      f(now, 1);
    }
  }

  // f(key) for every probability whose upper half this is.
  template <typename F>
  __device__ __forceinline__ void in_bin(uint32_t bin, int first, int step, F f) const {
    int i0 = begin + first;
    if (P.vec) {
      const int vecs = (end - begin) / 4;
      const uint4* p = reinterpret_cast<const uint4*>((const uint32_t*)row + begin);
      constexpr int kAhead = 4;
      for (int v = first; v < vecs; v += kAhead * step) {
        uint4 x[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
          if (v + k * step < vecs) x[k] = __ldg(p + v + k * step);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          if (v + k * step >= vecs) break;
          const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (w[j] >> 16 == bin) f(w[j]);
        }
      }
      i0 += vecs * 4;
    }
    for (int i = i0; i < end; i += step) {
      const uint32_t w = __ldg((const uint32_t*)row + i);
      if (w >> 16 == bin) f(w);
    }
  }

  // f(index) for every entry of the part with this (not zero) key, in any order.
  template <typename F>
  __device__ __forceinline__ void matches(uint32_t key, int first, int step, F f) const {
    constexpr int N = PROBS ? 4 : 8;
    int i0 = begin + first;
    if (P.vec) {
      const int vecs = (end - begin) / N;
      const uint4* p = reinterpret_cast<const uint4*>((const char*)row + (size_t)begin * (PROBS ? 4 : 2));
      // two logits at a time: the words' halves that are zero after the exclusive or
      const bool zero = !PROBS && key == 0x8000u;
      const uint32_t bits = PROBS ? key : (key & 0x8000u ? key & 0x7fffu : ~key & 0xffffu) * 0x10001u;
      const uint32_t mask = zero ? 0x7fff7fffu : 0xffffffffu;
      auto one = [&](const uint4& v, int at) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t hit = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (PROBS) {
            // (what is above 1 counts as 1)
            hit |= (key == 0x3f800000u ? prob_key(w[j]) : w[j]) == bits;
          } else {
            const uint32_t x = (w[j] & mask) ^ bits;
            hit |= (x - 0x00010001u) & ~x & 0x80008000u;
          }
        }
        if (hit)
          for (int j = 0; j < N; ++j)
            if (key_at(at + j) == key) f(at + j);
      };
      constexpr int kAhead = 4;
      for (int v = first; v < vecs; v += kAhead * step) {
        uint4 x[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
          if (v + k * step < vecs) x[k] = __ldg(p + v + k * step);
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
          if (v + k * step < vecs) one(x[k], begin + (v + k * step) * N);
      }
      i0 += vecs * N;
    }
    for (int i = i0; i < end; i += step)
      if (key_at(i) == key) f(i);
  }

  // out[index] = value(index, key) for every entry of the part.
  template <typename F>
  __device__ __forceinline__ void write(float* out, int vec_out, int first, int step, F value) const {
    constexpr int N = PROBS ? 4 : 8;
    if (!P.vec || !vec_out) {
      for (int i = begin + first; i < end; i += step) out[i] = value(i, key_at(i));
      return;
    }
    const int vecs = (end - begin) / N;
    const uint4* p = reinterpret_cast<const uint4*>((const char*)row + (size_t)begin * (PROBS ? 4 : 2));
#pragma unroll 2
    for (int v = first; v < vecs; v += step) {
      const uint4 x = __ldg(p + v);
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
      const int i = begin + v * N;
      float4* o = reinterpret_cast<float4*>(out + i);
      if (PROBS) {
        __stcs(o, make_float4(value(i, prob_key(w[0])), value(i + 1, prob_key(w[1])),
                              value(i + 2, prob_key(w[2])), value(i + 3, prob_key(w[3]))));
      } else {
#pragma unroll
        for (int q = 0; q < 2; ++q)
          __stcs(o + q, make_float4(value(i + 4 * q, logit_key(w[2 * q] & 0xffffu)),
                                    value(i + 4 * q + 1, logit_key(w[2 * q] >> 16)),
                                    value(i + 4 * q + 2, logit_key(w[2 * q + 1] & 0xffffu)),
                                    value(i + 4 * q + 3, logit_key(w[2 * q + 1] >> 16))));
      }
    }
    for (int i = begin + vecs * N + first; i < end; i += step) out[i] = value(i, key_at(i));
  }

  // f(index, key) for every entry of [a, b) that this thread takes, `step` vectors apart from `first`.
  template <typename F>
  __device__ __forceinline__ void each(int a, int b, int first, int step, F f) const {
    constexpr int N = PROBS ? 4 : 8;
    if (!P.vec) {
      for (int i = a + first; i < b; i += step) f(i, key_at(i));
      return;
    }
    const int vecs = (b - a) / N;
    const uint4* p = reinterpret_cast<const uint4*>((const char*)row + (size_t)a * (PROBS ? 4 : 2));
    auto one = [&](const uint4& v, int at) {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (PROBS) {
          f(at + j, prob_key(w[j]));
        } else {
          f(at + 2 * j, logit_key(w[j] & 0xffffu));
          f(at + 2 * j + 1, logit_key(w[j] >> 16));
        }
      }
    };
    int v = first;
    for (; v + 3 * step < vecs; v += 4 * step) {
      uint4 x[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = __ldg(p + v + k * step);
#pragma unroll
      for (int k = 0; k < 4; ++k) one(x[k], a + (v + k * step) * N);
    }
    for (; v < vecs; v += step) one(__ldg(p + v), a + v * N);
    for (int i = a + vecs * N + first; i < b; i += step) f(i, key_at(i));
  }
};

template <bool PROBS, bool WRITE>
__global__ void __launch_bounds__(kRowThreads, 1) rows_kernel(const RowsParams P) {
  extern __shared__ __align__(16) unsigned char s_hist[];
  __shared__ RowShared sh;
  uint32_t* hist = reinterpret_cast<uint32_t*>(s_hist);                       // logits: two counts
  unsigned long long* hist64 = reinterpret_cast<unsigned long long*>(s_hist);  // count << 40 | sum
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // (quick_kernel's marks; the launch overlaps its end)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  for (int row = blockIdx.x / C; row < P.n_rows; row += gridDim.x / C) {
  if (WRITE ? P.probs[(size_t)row * P.ld_out] != kMarkProb : P.tokens[row] != kMarkToken) continue;
  const int req = row / P.J;
  const float T = P.temperature ? P.temperature[req] : 1.f;
  const bool greedy = !(T > 0.f);
  const RowReader<PROBS> in{P, (const char*)P.rows + (size_t)row * P.ld * (PROBS ? 4 : 2),
                      min(P.V, rank * P.part), min(P.V, (rank + 1) * P.part)};

  // ---- 1. this CTA's histogram and largest key ----
  for (int i = tid; i < kHistBytes / 16; i += kRowThreads)
    reinterpret_cast<uint4*>(s_hist)[i] = make_uint4(0, 0, 0, 0);
  if (tid < 64) {
    const double t = exp2((double)tid / 64.0);
    const float hi = (float)t;
    sh.two_to[tid] = make_float2(hi, (float)(t - (double)hi));
  } else if (tid == 64 && !PROBS) {
    const double c = 1.4426950408889634074 / fmin(fmax((double)(greedy ? 1.f : T), 0x1p-100), 0x1p100);
    const float hi = (float)c;
    sh.per_unit = make_float2(hi, (float)(c - (double)hi));
  }
  if (tid == 65) sh.found = sh.inside = Border{0, 0, 0, 0, 0};
  cluster.sync();  // (every CTA has begun: its shared memory may be written from here on)
  uint32_t top = 0;
  in.each(in.begin, in.end, tid, kRowThreads, [&](int, uint32_t k) {
    if (!k) return;
    top = max(top, k);
    if (PROBS)  // (descending: bin 0 holds the largest; keys are at most 0x3f80 << 16)
      atomicAdd(&hist64[0x3fff - (k >> 16)], 1ull << 40 | (k & 0xffffu));
    else
      atomicAdd(&hist[0x7fff - (k >> 1)], k & 1 ? 1u : 65536u);
  });
  top = __reduce_max_sync(0xffffffffu, top);
  if (lane == 0) sh.warp_count[warp] = top;
  __syncthreads();
  if (warp == 0) {
    top = __reduce_max_sync(0xffffffffu, sh.warp_count[lane]);
    if (lane < C) cluster.map_shared_rank(sh.rank_top, lane)[rank] = top;
  }
  cluster.sync();
  top = 0;
  for (int c = 0; c < C; ++c) top = max(top, sh.rank_top[c]);

  // ---- 2. counts and sums before every row of 32 histogram words of this warp ----
  const float top_value = PROBS ? 0.f : logit_value(top);
  const int top_exp = PROBS ? max(1, (int)(top >> 23)) : 0;
  const float2 per_unit = sh.per_unit;
  // an entry's weight as a count of 2^-62 (logits)
  auto weight = [&](uint32_t k) -> unsigned long long {
    if (k == top) return 1ull << kSumBits;
    if (top == 0xff80u) return 0;  // beside +inf nothing weighs anything
    return weight62(ff_sum(logit_value(k), -top_value), per_unit, sh.two_to);
  };
  // exponent of a probability bin's (or key's) last place, relative to the units of the sums
  auto place = [&](uint32_t k) { return max(1, (int)(k >> 23)) - top_exp + kSumBits - 24; };
  auto bin_base = [&](uint32_t k) {  // the 24-bit significand with the lower 16 bits zero
    return ((k >> 23) ? 0x800000u : 0u) | (k & 0x7f0000u);
  };
  constexpr int kWords = PROBS ? kHistBytes / 8 : kHistBytes / 4;
  const int my_rows = kWords / 32 / (C * kRowWarps);
  const int word0 = (rank * kRowWarps + warp) * my_rows * 32;
  // the entries of this lane's word of a row: two values (logits), the larger first, or one bin
  struct Word {
    uint32_t n0, n1;
    u128 s0, s1;
    unsigned long long w0, w1;
  };
  auto read_word = [&](int word) {
    Word x = {0, 0, 0, 0, 0, 0};
    if (PROBS) {
      unsigned long long low = 0;
      for (int c = 0; c < C; ++c) {
        const unsigned long long v = *cluster.map_shared_rank(hist64 + word, c);
        x.n0 += (uint32_t)(v >> 40);
        low += v & 0xffffffffffull;
      }
      const uint32_t k = (uint32_t)(0x3fff - word) << 16;
      x.s0 = shifted((unsigned long long)x.n0 * bin_base(k) + low, place(k));
      x.w0 = low;
    } else {
      for (int c = 0; c < C; ++c) {
        const uint32_t v = *cluster.map_shared_rank(hist + word, c);
        x.n0 += v & 0xffffu;
        x.n1 += v >> 16;
      }
      const uint32_t k = (uint32_t)(0x7fff - word) * 2 + 1;
      if (x.n0) x.s0 = (u128)(x.w0 = weight(k)) * x.n0;
      if (x.n1) x.s1 = (u128)(x.w1 = weight(k - 1)) * x.n1;
    }
    return x;
  };
  uint32_t row_count = 0;           // lane i: of row i, then of the rows before it
  u128 row_sum = 0;
  for (int i = 0; i < my_rows; ++i) {
    const Word x = read_word(word0 + i * 32 + lane);
    const uint32_t n = __reduce_add_sync(0xffffffffu, x.n0 + x.n1);
    if (n) {
      const u128 s = warp_sum(x.s0 + x.s1);
      if (lane == i) {
        row_count = n;
        row_sum = s;
      }
    }
  }
  uint32_t count_at = warp_before(row_count);
  u128 sum_at = warp_before(row_sum);
  uint32_t my_count = from_lane(count_at + row_count, 31);
  u128 my_sum = from_lane(sum_at + row_sum, 31);
  if (lane == 0) {
    sh.warp_count[warp] = my_count;
    sh.warp_sum[warp] = my_sum;
  }
  __syncthreads();
  {
    const uint32_t n = sh.warp_count[lane];
    const u128 s = sh.warp_sum[lane];
    const uint32_t nb = warp_before(n);
    const u128 sb = warp_before(s);
    if (warp == 0) {
      const uint32_t all_n = from_lane(nb + n, 31);
      const u128 all_s = from_lane(sb + s, 31);
      if (lane < C) {
        cluster.map_shared_rank(sh.rank_count, lane)[rank] = all_n;
        cluster.map_shared_rank(sh.rank_sum, lane)[rank] = all_s;
      }
    }
    count_at += from_lane(nb, warp);
    sum_at += from_lane(sb, warp);
  }
  cluster.sync();
  uint32_t total = 0;
  u128 total_sum = 0;
  for (int c = 0; c < C; ++c) {
    if (c == rank) {
      count_at += total;
      sum_at += total_sum;
    }
    total += sh.rank_count[c];
    total_sum += sh.rank_sum[c];
  }
  const uint32_t count0 = from_lane(count_at, 0);  // before this warp
  const u128 sum0 = from_lane(sum_at, 0);

  // ---- 3. places in the order ----
  // By count: the entry at place g (from 0). By sum: the one whose stretch of the running sum holds place
  // at_sum. By key: the value `g`, whether it occurs or not. Every thread of the cluster calls this alike.
  enum { kByCount, kBySum, kByKey };
  auto find = [&](int by, uint32_t g, u128 at_sum) -> Border {
    const int key_word = by == kByKey ? (PROBS ? 0x3fff - (int)(g >> 16) : 0x7fff - (int)(g >> 1)) : 0;
    bool mine = by == kByCount ? g >= count0 && g - count0 < my_count
                : by == kBySum ? at_sum >= sum0 && at_sum - sum0 < my_sum
                               : key_word >= word0 && key_word < word0 + my_rows * 32;
    if (mine) {
      uint32_t at;
      if (by == kByKey) {
        at = (key_word - word0) >> 5;
      } else {
        const bool before = by == kByCount ? count_at <= g : sum_at <= at_sum;
        // (rows beyond this warp's, and empty ones, stand where the next one begins)
        at = 31 - __clz(__ballot_sync(0xffffffffu, before && lane < my_rows));
        // of rows that begin at the same place the last one is not empty
      }
      const uint32_t base_n = from_lane(count_at, at);
      const u128 base_s = from_lane(sum_at, at);
      const Word x = read_word(word0 + at * 32 + lane);
      const uint32_t n = base_n + warp_before(x.n0 + x.n1);
      const u128 s = base_s + warp_before(x.s0 + x.s1);
      bool here, second = false;
      if (by == kByCount) {
        here = g >= n && g < n + x.n0 + x.n1;
        second = g >= n + x.n0;
      } else if (by == kBySum) {
        here = at_sum >= s && at_sum < s + x.s0 + x.s1;
        second = at_sum >= s + x.s0;
      } else {
        here = word0 + (int)at * 32 + lane == key_word;
        second = !PROBS && !(g & 1);
      }
      if (here) {
        Border b;
        const int word = word0 + at * 32 + lane;
        b.key = PROBS ? (uint32_t)(0x3fff - word) << 16 : (uint32_t)(0x7fff - word) * 2 + (second ? 0 : 1);
        b.above = n + (second ? x.n0 : 0);
        b.count = second ? x.n1 : x.n0;
        b.sum = s + (second ? x.s0 : 0);
        b.w = second ? x.w1 : x.w0;
        for (int c = 0; c < C; ++c) *cluster.map_shared_rank(&sh.found, c) = b;
      }
    }
    cluster.sync();
    Border b = sh.found;
    cluster.sync();
    if (!PROBS) return b;
    // A probability's bin holds 65536 values: two passes over the row find the one in question.
    const int up = place(b.key);
    auto one = [&](uint32_t k) {
      return (unsigned long long)shifted(bin_base(k) | (k & 0xffffu), up);
    };
    if (b.count == 1 && by != kByKey) {
      b.key |= (uint32_t)b.w;  // the sum of the lower halves is that of the only entry
      b.w = one(b.key);
      return b;
    }
    for (int level = 0; level < 2; ++level) {
      const int shift = level ? 0 : 8;
      if (tid < 256) {
        sh.low[tid] = 0;
        sh.low_sum[tid] = 0;
      }
      __syncthreads();
      const uint32_t want = b.key >> (shift + 8);
      in.each(in.begin, in.end, tid, kRowThreads, [&](int, uint32_t k) {
        if (k >> (shift + 8) != want) return;
        atomicAdd(&sh.low[255 - ((k >> shift) & 255u)], 1u);
        if (!level) atomicAdd(&sh.low_sum[255 - ((k >> 8) & 255u)], (unsigned long long)(k & 255u));
      });
      cluster.sync();
      uint32_t n = 0, before_n = 0;
      unsigned long long s = 0, before_s = 0;
      const uint32_t key = b.key | (255u - (uint32_t)tid) << shift;
      if (tid < 256) {
        for (int c = 0; c < C; ++c) {
          n += *cluster.map_shared_rank(&sh.low[tid], c);
          s += *cluster.map_shared_rank(&sh.low_sum[tid], c);
        }
        s += (unsigned long long)n * (bin_base(key) | (key & 0xffffu));
        before_n = warp_before(n);
        before_s = warp_before(s);
        if (lane == 31) {
          sh.merged[warp] = before_n + n;
          sh.merged_sum[warp] = before_s + s;
        }
      }
      __syncthreads();
      if (tid < 256) {
        for (int w = 0; w < warp; ++w) {
          before_n += sh.merged[w];
          before_s += sh.merged_sum[w];
        }
        const u128 from = b.sum + shifted(before_s, up), to = b.sum + shifted(before_s + s, up);
        bool here;
        if (by == kByCount) {
          here = g >= b.above + before_n && g < (unsigned long long)b.above + before_n + n;
        } else if (by == kBySum) {
          // (the bin's own sum may have been rounded: what lies past its last entry is the last entry's)
          here = n > 0 && (at_sum >= from || before_n == 0) && (at_sum < to || before_n + n == b.count);
        } else {
          here = (uint32_t)(g >> shift) == key >> shift;
        }
        if (here)
          sh.inside = Border{key, b.above + before_n, n, level ? one(key) : 0, from};
      }
      cluster.sync();
      b = sh.inside;
      __syncthreads();
    }
    return b;
  };

  if (total == 0) {
    if (rank == 0 && tid == 0) {
      raise_err(P.err, SD_ERR_ZERO_ROW);
      if (P.kept) P.kept[row] = 0;
      if (!WRITE) {
        P.tokens[row] = 0;
        if (P.prob) P.prob[row] = 0.f;
      }
    }
    if (WRITE)
      for (int i = in.begin + tid; i < in.end; i += kRowThreads) P.probs[(size_t)row * P.ld_out + i] = 0.f;
    cluster.sync();
    continue;
  }

  // The last entry kept, and the sum of those kept.
  uint32_t n = total;
  Border last = {0, 0, 0, 0, 0};
  bool cut = false;
  u128 kept_sum = total_sum;
  auto cut_at = [&](uint32_t m, const Border& b) {
    n = m;
    last = b;
    cut = true;
    kept_sum = b.sum + (u128)b.w * (m - b.above);
  };
  uint32_t k = 0x7fffffffu;
  if (P.top_k && P.top_k[req] > 0) k = (uint32_t)P.top_k[req];
  if (!PROBS && top == 0xff80u) k = min(k, find(kByKey, top, 0).count);
  if (greedy) k = 1;
  if (k < n) cut_at(k, find(kByCount, k - 1, 0));
  const float top_p = P.top_p && !greedy ? P.top_p[req] : 1.f;
  if (top_p < 1.f && n > 1) {
    // the last entry before which less than top_p of the sum lies
    const u128 at = last_place(top_p, kept_sum, total_sum);
    const Border b = find(kBySum, 0, at);
    const uint32_t m = b.above + 1 + quotient(at > b.sum ? at - b.sum : 0, b.w, b.count - 1);
    if (m < n) cut_at(m, b);
  }
  const float min_p = P.min_p && !greedy ? P.min_p[req] : 0.f;
  if (min_p > 0.f && n > 1) {
    uint32_t m;
    if (min_p >= 1.f) {
      m = find(kByKey, top, 0).count;
    } else if (PROBS) {
      const float t = __double2float_ru((double)min_p * (double)__uint_as_float(top));
      const Border b = find(kByKey, max(1u, __float_as_uint(t)), 0);
      m = b.above + b.count;
    } else {
      const uint32_t key = least_logit_key(top_value, T, min_p);
      const Border b = find(kByKey, min(max(key, 0x80u), top), 0);
      m = b.above + b.count;
    }
    m = max(m, 1u);
    if (m < n) cut_at(m, find(kByCount, m - 1, 0));
  }
  if (rank == 0 && tid == 0 && P.kept) P.kept[row] = (int32_t)n;

  // ---- 4. the entry in question among those of its value, by index ----
  // Index of entry number j (from 0) of those with this key. A warp goes over a stretch of its own.
  auto nth = [&](uint32_t key, uint32_t j) -> int {
    const int len = in.end - in.begin, seg = ((len + kRowWarps - 1) / kRowWarps + 7) & ~7;
    const int a = in.begin + min(len, warp * seg), b = in.begin + min(len, (warp + 1) * seg);
    uint32_t have = 0;
    in.each(a, b, lane, 32, [&](int, uint32_t x) { have += x == key; });
    have = __reduce_add_sync(0xffffffffu, have);
    if (lane == 0) sh.warp_count[warp] = have;
    __syncthreads();
    const uint32_t v = sh.warp_count[lane];
    const uint32_t vb = warp_before(v);
    if (warp == 0) {
      const uint32_t all = __shfl_sync(0xffffffffu, vb + v, 31);
      if (lane < C) cluster.map_shared_rank(sh.rank_eq, lane)[rank] = all;
    }
    uint32_t before = __shfl_sync(0xffffffffu, vb, warp);
    cluster.sync();
    for (int c = 0; c < rank; ++c) before += sh.rank_eq[c];
    if (j >= before && j - before < have) {
      uint32_t left = j - before;
      for (int i = a; i < b; i += 32) {
        const uint32_t m = __ballot_sync(0xffffffffu, i + lane < b && in.key_at(i + lane) == key);
        const uint32_t c = __popc(m);
        if (left < c) {
          const int at = i + (int)__fns(m, 0, (int)left + 1);
          if (lane < C) *cluster.map_shared_rank(&sh.index, lane) = at;
          break;
        }
        left -= c;
      }
    }
    cluster.sync();
    return sh.index;
  };

  if (!WRITE) {
    Border b;
    uint32_t j = 0;
    if (n == 1) {
      b = cut ? last : find(kByCount, 0, 0);
    } else {
      const u128 at = draw_place(P.u[row], kept_sum, total_sum);
      b = find(kBySum, 0, at);
      j = quotient(at > b.sum ? at - b.sum : 0, b.w, b.count - 1);
      if (b.above + j >= n) {
        b = cut ? last : find(kByCount, n - 1, 0);
        j = n - 1 - b.above;
      }
    }
    const int at = nth(b.key, j);
    if (rank == 0 && tid == 0) {
      P.tokens[row] = at;
      if (P.prob) P.prob[row] = (float)((double)b.w / sum_double(kept_sum));
    }
  } else {
    int edge = 0x7fffffff;  // entries of the last value are kept up to here
    if (cut && n - last.above < last.count) edge = nth(last.key, n - last.above - 1);
    const uint32_t least = cut ? last.key : 1u;
    const KeptValue v = {pair_of(kSumUnit / sum_double(kept_sum)), per_unit, top_value,
                         PROBS ? __uint_as_float((uint32_t)(127 + 126 - top_exp) << 23) : 1.f};
    float* out = P.probs + (size_t)row * P.ld_out;
    auto value = [&](int i, uint32_t x) {
      // (of entries beside +inf only those that are +inf are kept)
      return x < least || (x == least && i > edge) ? 0.f : !PROBS && x == top ? v.inv.x : v.of<PROBS>(x);
    };
    in.write(out, P.vec_out, tid, kRowThreads, value);
  }
  cluster.sync();  // no CTA goes on while another may read its histogram
  }
}

// ---------------------------------------------------------------------------------------------
// The quick kernel. Bins stand in the order of the values, larger first, as rows of 32 (a lane a bin):
// logits have 128 rows of positive values, one for zero, 128 of negative ones; probabilities 256.
//
// Where a row's time goes (one token of each of 608 rows of 201088 logits, 4 CTAs of 256 threads an SM: 120
// us a row, 190 for the slowest): reading and counting 57 us (8 instructions an entry; a shared atomic of
// 32 different addresses takes 2.5 cycles), the sums of the bins 14, the search 11, the drawn value's
// entries 34: 608 rows do not stay in L2, so they come from memory a second time. 1024 rows are two rounds
// of those places, 340 us against 61 of memory. 2048 rows of logits cut: 974 us against 364; 384 of
// probabilities 464 against 91 (each place that is looked for reads the row again). One row of 1024: 27
// us, latency.
// ---------------------------------------------------------------------------------------------
constexpr int kQThreads = 256, kQWarps = kQThreads / 32, kQBins = 8192, kQRows = 257;
constexpr uint16_t kLeast = 0xc7ff;  // the least logit that has a counter, -130560
constexpr int kQSmall = 256;    // logits below 2^-15 that a CTA may have
constexpr int kQList = 2048;    // entries of one bin of probabilities

enum { kOpEnd, kOpNth, kOpCollect, kOpCount, kOpMark, kOpNothing };

// (At most 16 KB: four CTAs with their counters in 196 KB leave 60 KB of L1 for the row's second reading.
// With 17 KB, and so 28 KB of L1, that takes 80000 cycles a row instead of 70000.)
struct QuickShared {
  float2 two_to[64];
  uint32_t row_count[kQRows];  // of a row of bins, then of those before it (rank 0's)
  u128 row_sum[kQRows];
  int n_todo;
  uint32_t rank_first[kMostClusters];  // the first bin in order that a CTA has anything in
  uint32_t rank_zero[kMostClusters], rank_small[kMostClusters], rank_far[kMostClusters],
      rank_bad[kMostClusters];
  unsigned long long rank_small_sum[kMostClusters];  // (of 256 weights at most, in units of 2^-54)
  uint32_t zero, small, far, bad, first, eq[kQWarps];
  unsigned long long small_sum;
  float2 per_unit;
  // of rank 0's first warp to all: what to do, and the row's cut
  int op;
  uint32_t op_key, op_number, op_count;
  int index, edge;
  uint32_t least;
  float2 inv;
  // a bin's entries (lower halves), and counts and sums of them
  uint32_t listed;
  union {
    uint16_t list[kQList];
    int at[kQList];  // or indices of entries of one value
    struct {         // or, before the search, which rows of bins hold anything, and the small logits
      uint8_t filled[kQThreads];
      uint16_t todo[kQRows];
      uint16_t small_at[kQSmall];
    };
  };
  uint32_t sub[256], sub_sum[256];
};

// Bits of a logit by its place in the bins' order: row 128 is zero.
__device__ __forceinline__ uint32_t quick_bits(int row, int lane) {
  if (row == 128) return 0;
  const int i = row < 128 ? 4095 - (row * 32 + lane) : (row - 129) * 32 + lane;
  return (row < 128 ? 0u : 0x8000u) | (uint32_t)(0x4000 + i - 0x800);
}
// Its counter: the lower 12 bits and the sign above them. (Exponents of 2^-15 to 2^16 are those whose
// upper bit differs from the three below it, so that the lower 12 bits and the sign say it all; the
// fourth of them, upside down, is the value's order.)
__device__ __forceinline__ int quick_slot(uint32_t bits) {
  return (int)((bits & 0xfffu) | (bits >> 3 & 0x1000u));
}
__device__ __forceinline__ bool quick_has(uint32_t bits) {
  return ((bits ^ bits << 1) & 0x7000u) == 0x4000u;
}

static_assert(sizeof(QuickShared) <= 16384, "shared memory of four CTAs");

template <bool PROBS, bool WRITE>
__global__ void __launch_bounds__(kQThreads, PROBS ? 3 : 4) quick_kernel(const RowsParams P) {
  extern __shared__ __align__(16) unsigned char s_hist[];
  __shared__ QuickShared sh;
  uint32_t* count = reinterpret_cast<uint32_t*>(s_hist);  // probabilities: then sums of the lower halves
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // (the search and those that serve it meet from different places of the program, which __syncthreads and
  // a group's sync do not allow: barriers that count warps and threads)
  auto meet = [&]() {
    if (C == 1) named_bar(1, kQThreads);
    else asm volatile("barrier.cluster.arrive.release;\n barrier.cluster.wait.acquire;" ::: "memory");
  };
  const int row = blockIdx.x / C, req = row / P.J;
  const float T = P.temperature ? P.temperature[req] : 1.f;
  const bool greedy = !(T > 0.f);
  const RowReader<PROBS> in{P, (const char*)P.rows + (size_t)row * P.ld * (PROBS ? 4 : 2),
                            min(P.V, rank * P.part), min(P.V, (rank + 1) * P.part)};

  // ---- 1. this CTA's histogram ----
  for (int i = tid; i < kQBins * (PROBS ? 2 : 1) / 4; i += kQThreads)
    reinterpret_cast<uint4*>(s_hist)[i] = make_uint4(0, 0, 0, 0);
  if (!PROBS && tid < 64) {
    const double t = exp2((double)tid / 64.0);
    const float hi = (float)t;
    sh.two_to[tid] = make_float2(hi, (float)(t - (double)hi));
  } else if (!PROBS && tid == 64) {
    const double c = 1.4426950408889634074 / fmin(fmax((double)(greedy ? 1.f : T), 0x1p-100), 0x1p100);
    const float hi = (float)c;
    sh.per_unit = make_float2(hi, (float)(c - (double)hi));
  } else if (tid == 96) {
    sh.zero = sh.small = sh.far = sh.bad = 0;
    sh.first = 0xffffffffu;
    sh.small_sum = 0;
  }
  meet();  // (every CTA has begun: its shared memory may be written from here on)
  {
    uint32_t zeros = 0, far = 0, bad = 0, largest = 0;
    char* at = reinterpret_cast<char*>(count);
    auto odd_logit = [&](uint32_t b) {  // one of magnitude below 2^-15
      if ((b & 0x7fffu) == 0) {
        ++zeros;
      } else {
        const uint32_t i = atomicAdd(&sh.small, 1u);
        if (i < kQSmall) sh.small_at[i] = (uint16_t)b;
      }
    };
    // Logits of -2^17 and less, -inf and NaN become the least that has a counter, and are told apart
    // only if it matters how many there are. One above 2^17 shows in the maximum.
    __nv_bfloat162 most = __halves2bfloat162(__ushort_as_bfloat16(kLeast), __ushort_as_bfloat16(kLeast));
    const __nv_bfloat162 least2 = most;
    in.raw(tid, kQThreads, [&](const uint32_t (&w)[4], int n) {
      if (PROBS) {
        bool odd = false;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (j && n == 1) break;
          if (w[j] >> 29 == 1) {
            uint32_t* c = reinterpret_cast<uint32_t*>(at + (w[j] >> 14 & 0x7ffcu));
            atomicAdd(c, 1u);
            atomicAdd(c + kQBins, w[j] & 0xffffu);
            largest = max(largest, w[j]);
          } else {
            odd |= w[j] != 0;
          }
        }
        if (odd)
          for (int j = 0; j < 4; ++j) {
            if (j && n == 1) break;
            if (w[j] - 1u < 0x1fffffffu) ++far;  // below 2^-63
            else if (w[j] >> 29 != 1 && w[j] - 1u < 0x7f800000u) bad = 1;
          }
      } else {
        uint32_t v[4], odd = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const __nv_bfloat162 x = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&w[j]), least2);
          most = __hmax2(most, x);
          v[j] = *reinterpret_cast<const uint32_t*>(&x);
          odd |= ((v[j] ^ v[j] << 1) & 0x70007000u) ^ 0x40004000u;
        }
        if (n == 1) {  // (its word's upper half is no entry)
          if (quick_has(v[0] & 0xffffu)) atomicAdd(&count[quick_slot(v[0] & 0xffffu)], 1u);
          else odd_logit(v[0] & 0xffffu);
        } else if (!odd) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            atomicAdd(reinterpret_cast<uint32_t*>(at + ((v[j] << 2 & 0x3ffcu) | (v[j] >> 1 & 0x4000u))), 1u);
            atomicAdd(reinterpret_cast<uint32_t*>(at + ((v[j] >> 14 & 0x3ffcu) | (v[j] >> 17 & 0x4000u))), 1u);
          }
        } else {
          for (int j = 0; j < 8; ++j) {
            const uint32_t b = j & 1 ? v[j >> 1] >> 16 : v[j >> 1] & 0xffffu;
            if (quick_has(b)) atomicAdd(&count[quick_slot(b)], 1u);
            else if ((b & 0x7fffu) < 0x3800u) odd_logit(b);
          }
        }
      }
    });
    if (largest > 0x3f800000u) bad = 1;
    if (!PROBS && (__low2float(most) >= 131072.f || __high2float(most) >= 131072.f)) bad = 1;
    zeros = __reduce_add_sync(0xffffffffu, zeros);
    far = __reduce_add_sync(0xffffffffu, far);
    bad = __reduce_or_sync(0xffffffffu, bad);
    if (lane == 0) {
      if (zeros) atomicAdd(&sh.zero, zeros);
      if (far) atomicAdd(&sh.far, far);
      if (bad) sh.bad = 1;
    }
  }
  __syncthreads();
  if (!PROBS && tid == 0) {
    sh.far = count[quick_slot(kLeast)];
    count[quick_slot(kLeast)] = 0;
  }
  __syncthreads();
  // the first bin in order that is not empty
  {
    uint32_t first = 0xffffffffu;
    constexpr int kPer = kQBins / kQThreads;
    const uint4* c4 = reinterpret_cast<const uint4*>(count) + tid * (kPer / 4);
    uint32_t some = 0;
#pragma unroll
    for (int i = 0; i < kPer / 4; ++i) {
      const uint4 v = c4[i];
      some |= (v.x ? 1u : 0u) << (4 * i) | (v.y ? 2u : 0u) << (4 * i) | (v.z ? 4u : 0u) << (4 * i) |
              (v.w ? 8u : 0u) << (4 * i);
      if (PROBS && (v.x | v.y | v.z | v.w) > 0xffffu) sh.bad = 1;  // sums of 16 bits may have passed 32
    }
    sh.filled[tid] = some != 0;
    if (some) {
      // counters ascend with the magnitude; zero is place 4096, negative logits follow
      const int at = PROBS ? tid * kPer : tid * kPer ^ 0x800;
      if (PROBS) first = 8191 - (at + 31 - __clz(some));
      else if (at < 4096) first = 4095 - (at + 31 - __clz(some));
      else first = 1 + at + __ffs(some) - 1;
    }
    if (!PROBS && tid == 0 && sh.zero + sh.small) first = min(first, 4096u);
    first = __reduce_min_sync(0xffffffffu, first);
    if (lane == 0) atomicMin(&sh.first, first);
  }
  __syncthreads();
  if (warp == 0 && lane < C) {
    cluster.map_shared_rank(sh.rank_first, lane)[rank] = sh.first;
    cluster.map_shared_rank(sh.rank_zero, lane)[rank] = sh.zero;
    cluster.map_shared_rank(sh.rank_small, lane)[rank] = sh.small;
    cluster.map_shared_rank(sh.rank_far, lane)[rank] = sh.far;
    cluster.map_shared_rank(sh.rank_bad, lane)[rank] =
        sh.bad | (uint32_t)(sh.small > kQSmall ? 1 : 0);
  }
  meet();
  uint32_t first = 0xffffffffu, zeros = 0, smalls = 0, far = 0, bad = 0;
  for (int c = 0; c < C; ++c) {
    first = min(first, sh.rank_first[c]);
    zeros += sh.rank_zero[c];
    smalls += sh.rank_small[c];
    far += sh.rank_far[c];
    bad |= sh.rank_bad[c];
  }
  const bool some = first != 0xffffffffu;
  // the largest logit (some small one, if there is none above: such rows are marked)
  const uint32_t top_bits = !PROBS && some
      ? first == 4096 ? 0u : first < 4096 ? quick_bits(first >> 5, first & 31)
                                          : quick_bits(129 + ((first - 4097) >> 5), (first - 4097) & 31)
      : 0u;
  const float top_value = bf16_bits_to_float(top_bits);
  const float2 per_unit = sh.per_unit;
  // a logit's weight as a count of 2^-62
  auto weight = [&](uint32_t bits) -> unsigned long long {
    if (bits == top_bits) return 1ull << kSumBits;
    return weight62(ff_sum(bf16_bits_to_float(bits), -top_value), per_unit, sh.two_to);
  };
  // a bin's entries (and, of probabilities, the sum of their lower halves)
  auto count_of = [&](int r, unsigned long long& lows) -> uint32_t {
    uint32_t n = 0;
    lows = 0;
    if (!PROBS && r == 128) return lane == 0 ? zeros : 0;
    const int at = PROBS ? 8191 - (r * 32 + lane) : quick_slot(quick_bits(r, lane));
    if (C == 1) {
      n = count[at];
      if (PROBS) lows = count[at + kQBins];
    } else {
      for (int c = 0; c < C; ++c) {
        const uint32_t* from = cluster.map_shared_rank(count + at, c);
        n += from[0];
        if (PROBS) lows += from[kQBins];
      }
    }
    return n;
  };
  // their sum; w: the weight of each (logits)
  auto bin_sum = [&](int r, uint32_t n, unsigned long long lows, unsigned long long& w) -> u128 {
    if (!PROBS) return (u128)(w = weight(quick_bits(r, lane))) * n;
    if (n == 0) return 0;
    const uint32_t k = (uint32_t)(0x3fff - (r * 32 + lane));
    const unsigned long long units = (unsigned long long)n * ((0x80u | (k & 0x7fu)) << 16) + lows;
    // (the significand's last place, in units of 2^-62)
    return shifted(units, (int)(k >> 7) - 150 + kSumBits);
  };

  // ---- 2. counts and sums of the rows of bins, into rank 0 ----
  if (!PROBS) {  // small logits weigh for themselves, and stand beside zero
    unsigned long long s = 0;
    const uint32_t m = min(sh.small, (uint32_t)kQSmall);
    if ((uint32_t)tid < m) s = ((weight(sh.small_at[tid]) >> 7) + 1) >> 1;
    if (m) {
      s = (unsigned long long)warp_sum(s);
      if (lane == 0 && s) atomicAdd(&sh.small_sum, s);
    }
    __syncthreads();
    if (tid == 0) cluster.map_shared_rank(sh.rank_small_sum, 0)[rank] = sh.small_sum;
  }
  constexpr int kRowsOf = PROBS ? 256 : 257, kTogether = 2;
  // A CTA alone has noted which of its rows are empty (its threads looked at one each).
  auto filled = [&](int r) {
    if (C > 1 || (!PROBS && r == 128)) return true;
    return (bool)sh.filled[PROBS ? 255 - r : (r < 128 ? 127 - r : r - 1) ^ 64];
  };
  if (C == 1) {
    if (warp == 0) {  // the others, one behind another
      int n = 0;
      for (int r0 = 0; r0 < kRowsOf; r0 += 32) {
        const int r = r0 + lane;
        const bool take = r < kRowsOf && filled(r);
        const uint32_t m = __ballot_sync(0xffffffffu, take);
        if (take) sh.todo[n + __popc(m & ((1u << lane) - 1))] = (uint16_t)r;
        else if (r < kRowsOf) {
          sh.row_count[r] = 0;
          sh.row_sum[r] = 0;
        }
        n += __popc(m);
      }
      if (lane == 0) sh.n_todo = n;
    }
    __syncthreads();
  }
  const int rows_todo = C == 1 ? sh.n_todo : kRowsOf;
  for (int i0 = rank * kQWarps + warp; i0 < rows_todo; i0 += kTogether * C * kQWarps) {
    uint32_t n[kTogether];
    unsigned long long low[kTogether], w;
    u128 s[kTogether];
    int r[kTogether];
    bool any = false;
#pragma unroll
    for (int k = 0; k < kTogether; ++k) {
      const int i = i0 + k * C * kQWarps;
      r[k] = i < rows_todo ? C == 1 ? sh.todo[i] : i : -1;
      n[k] = 0;
      s[k] = low[k] = 0;
      if (r[k] >= 0) n[k] = count_of(r[k], low[k]);
      any |= n[k] != 0;
    }
    if (__any_sync(0xffffffffu, any)) {
#pragma unroll
      for (int k = 0; k < kTogether; ++k) s[k] = bin_sum(max(r[k], 0), n[k], low[k], w);
    }
#pragma unroll
    for (int k = 0; k < kTogether; ++k) {
      const uint32_t all = __reduce_add_sync(0xffffffffu, n[k]);
      if (all) s[k] = warp_sum(s[k]);
      if (lane == 0 && r[k] >= 0) {
        QuickShared* s0 = C == 1 ? &sh : cluster.map_shared_rank(&sh, 0);
        s0->row_count[r[k]] = all;
        s0->row_sum[r[k]] = all ? s[k] : (u128)0;
      }
    }
  }
  meet();

  // ---- 3. the search: rank 0's first warp, the others serve it ----
  float* out = WRITE ? P.probs + (size_t)row * P.ld_out : nullptr;
  const int worker = tid - (rank ? 0 : 32), workers = kQThreads - (rank ? 0 : 32);
  // Index of entry number op_number of those with op_key: up to kQList of them are listed and the
  // one with so many smaller ones is found; more are counted along the row.
  auto nth = [&]() {
    QuickShared* s0 = cluster.map_shared_rank(&sh, 0);
    const uint32_t key = s0->op_key, j = s0->op_number;
    if (s0->op_count <= kQList) {
      in.matches(key, worker, workers, [&](int i) { s0->at[atomicAdd(&s0->listed, 1u)] = i; });
      meet();
      if (rank == 0) {
        const int m = (int)sh.listed;
        for (int a = worker; a < m; a += workers) {
          const int mine = sh.at[a];
          uint32_t less = 0;
          for (int i = 0; i < m; ++i) less += sh.at[i] < mine;
          if (less == j) sh.index = mine;
        }
      }
      return;
    }
    const int w0 = worker >> 5, len = in.end - in.begin;
    const int seg = ((len + workers / 32 - 1) / (workers / 32) + 7) & ~7;
    const int a = in.begin + min(len, w0 * seg), b = in.begin + min(len, (w0 + 1) * seg);
    uint32_t have = 0;
    in.each(a, b, lane, 32, [&](int, uint32_t x) { have += x == key; });
    have = __reduce_add_sync(0xffffffffu, have);
    if (lane == 0) sh.eq[w0] = have;
    meet();
    uint32_t before = 0;
    for (int c = 0; c <= rank; ++c)
      for (int w = 0; w < (c == rank ? w0 : c ? kQWarps : kQWarps - 1); ++w)
        before += cluster.map_shared_rank(&sh, c)->eq[w];
    if (j >= before && j - before < have) {
      uint32_t left = j - before;
      for (int i = a; i < b;) {  // 256 entries at a time, then the 32 with the one in question
        uint32_t x[8], n = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = i + k * 32 + lane < b ? in.key_at(i + k * 32 + lane) : 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) n += __popc(__ballot_sync(0xffffffffu, x[k] == key));
        if (left >= n) {
          left -= n;
          i += 256;
          continue;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t m = __ballot_sync(0xffffffffu, x[k] == key), c = __popc(m);
          if (left < c && n) {
            if (lane == 0) s0->index = i + k * 32 + (int)__fns(m, 0, (int)left + 1);
            n = 0;
          } else if (n) {
            left -= c;
          }
        }
        break;
      }
    }
  };
  auto serve = [&]() {
    for (;;) {
      meet();
      QuickShared* s0 = cluster.map_shared_rank(&sh, 0);
      const int op = s0->op;
      if (op == kOpNth) {
        nth();
      } else if (op == kOpCollect) {  // the lower halves of a bin's entries
        in.in_bin(s0->op_key >> 16, worker, workers, [&](uint32_t x) {
          const uint32_t i = atomicAdd(&s0->listed, 1u);
          if (i < kQList) s0->list[i] = (uint16_t)x;
        });
      } else if (op == kOpCount) {  // the logits without a counter below that are numbers
        uint32_t n = 0;
        in.each(in.begin, in.end, worker, workers,
                [&](int, uint32_t x) { n += x && x <= logit_key(kLeast); });
        n = __reduce_add_sync(0xffffffffu, n);
        if (lane == 0 && n) atomicAdd(&s0->listed, n);
      } else {
        break;
      }
      meet();
    }
  };
  if (rank == 0 && warp == 0) {
    // counts and sums before every row
    constexpr int kPer = (kQRows + 31) / 32;
    uint32_t n = 0;
    u128 s = 0;
    if (!PROBS) {
      for (int c = 0; c < C; ++c) s += sh.rank_small_sum[c];
      if (lane == 0) {
        sh.row_count[128] += smalls;
        sh.row_sum[128] += s << 8;
      }
      s = 0;
      __syncwarp();
    }
    for (int i = 0; i < kPer; ++i)
      if (lane * kPer + i < kRowsOf) {
        n += sh.row_count[lane * kPer + i];
        s += sh.row_sum[lane * kPer + i];
      }
    uint32_t n_at = warp_before(n);
    u128 s_at = warp_before(s);
    const uint32_t binned = from_lane(n_at + n, 31);
    const u128 total_sum = from_lane(s_at + s, 31);
    for (int i = 0; i < kPer; ++i)
      if (lane * kPer + i < kRowsOf) {
        const uint32_t a = sh.row_count[lane * kPer + i];
        const u128 b = sh.row_sum[lane * kPer + i];
        sh.row_count[lane * kPer + i] = n_at;
        sh.row_sum[lane * kPer + i] = s_at;
        n_at += a;
        s_at += b;
      }
    __syncwarp();
    const uint32_t total = binned + far;
    // far entries have to weigh nothing beside the others
    bool mark = bad;
    if (PROBS) mark |= total > 0 && total_sum < (u128)1 << (kSumBits - 1);
    else if (far) mark |= !some || !((-130560.f - top_value) * per_unit.x < -64.f);
    if (!PROBS && some && first == 4096 && smalls) mark = true;

    auto ask = [&](int op, uint32_t key, uint32_t number, uint32_t of) {
      if (lane == 0) {
        sh.op = op;
        sh.op_key = key;
        sh.op_number = number;
        sh.op_count = of;
        sh.listed = 0;
      }
      meet();
      if (op == kOpNth) meet();  // (nth's own)
      if (op == kOpNth || op == kOpCollect || op == kOpCount) meet();
    };
    uint32_t listed_bin = 0;
    // A probability's place in its bin: by count (g), by sum (at_sum), or by key.
    auto inside = [&](Border b, int by, uint32_t g, u128 at_sum, uint32_t key) -> Border {
      const int up = (int)(b.key >> 23) - 150 + kSumBits;  // of its last place, in units of the sums
      auto one = [&](uint32_t k) {
        return (unsigned long long)shifted(0x800000u | (k & 0x7fffffu), up);
      };
      if (b.count == 1 && by != 2) {
        b.key |= (uint32_t)b.w;
        b.w = one(b.key);
        return b;
      }
      // (the last bin's entries are still listed, if it was this one)
      if (b.key != listed_bin) ask(kOpCollect, b.key, 0, b.count);
      listed_bin = b.key;
      const uint32_t m = sh.listed;
      if (m > kQList) {
        mark = true;
        return b;
      }
      for (int level = 0; level < 2; ++level) {
        // how far behind the sum before the bin the place lies, in the bin's last places
        const u128 d = at_sum > b.sum ? at_sum - b.sum : 0;
        const unsigned long long behind = (unsigned long long)(up >= 0 ? d >> up : d << -up);
        for (int i = lane; i < 256; i += 32) sh.sub[i] = sh.sub_sum[i] = 0;
        __syncwarp();
        for (uint32_t i = lane; i < m; i += 32) {
          const uint32_t x = sh.list[i];
          if (level && (x >> 8) != (b.key >> 8 & 0xffu)) continue;
          atomicAdd(&sh.sub[255 - (level ? x & 255u : x >> 8)], 1u);
          if (!level) atomicAdd(&sh.sub_sum[255 - (x >> 8)], x & 255u);
        }
        __syncwarp();
        // 8 bins a lane
        uint32_t bn = 0;
        unsigned long long bsum = 0;
        auto value = [&](int i) {
          return b.key | (uint32_t)(255 - i) << (level ? 0 : 8);
        };
        auto units = [&](int i) {
          return (unsigned long long)sh.sub[i] * (0x800000u | (value(i) & 0x7fffffu)) + sh.sub_sum[i];
        };
        for (int i = lane * 8; i < lane * 8 + 8; ++i) {
          bn += sh.sub[i];
          bsum += units(i);
        }
        uint32_t an = warp_before(bn);
        unsigned long long as = warp_before(bsum);
        bool hit = false;
        Border got = b;
        for (int i = lane * 8; i < lane * 8 + 8; ++i) {
          const uint32_t c = sh.sub[i];
          const unsigned long long u = units(i);
          bool here;
          if (by == 0) here = g >= b.above + an && g < (unsigned long long)b.above + an + c;
          else if (by == 1)
            here = c > 0 && (behind >= as || an == 0) && (behind < as + u || an + c == b.count);
          else here = (level ? key : key >> 8) == (level ? value(i) : value(i) >> 8);
          if (here) {
            hit = true;
            got = Border{value(i), b.above + an, c, one(value(i)), b.sum + shifted(as, up)};
          }
          an += c;
          as += u;
        }
        const uint32_t who = __ballot_sync(0xffffffffu, hit);
        const int src = who ? __ffs(who) - 1 : 0;
        b.key = __shfl_sync(0xffffffffu, got.key, src);
        b.above = __shfl_sync(0xffffffffu, got.above, src);
        b.count = __shfl_sync(0xffffffffu, got.count, src);
        b.sum = from_lane(got.sum, src);
        b.w = __shfl_sync(0xffffffffu, got.w, src);
        __syncwarp();
      }
      return b;
    };
    // The entry at place g of the order (by 0), the one whose stretch of the running sum holds place at_sum
    // (by 1), or a value, whether it occurs or not (by 2; g its place among the bins).
    auto find = [&](int by, uint32_t g, u128 at_sum, uint32_t key) -> Border {
      Border b = {0, 0, 1, 1, 0};
      if (by == 0 && g >= binned) {
        mark = true;
        return b;
      }
      int r;
      if (by == 2) {
        r = (int)(g >> 5);
      } else {
        int lo = 0, hi = kRowsOf;  // the last row that begins at g or before
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (by == 0 ? sh.row_count[mid] <= g : sh.row_sum[mid] <= at_sum) lo = mid;
          else hi = mid;
        }
        r = lo;
      }
      if (!PROBS && r == 128 && smalls) {
        mark = true;
        return b;
      }
      unsigned long long lows, w = 0;
      const uint32_t n = count_of(r, lows);
      const u128 s = bin_sum(r, n, lows, w);
      if (PROBS) w = lows;
      const uint32_t an = sh.row_count[r] + warp_before(n);
      const u128 as = sh.row_sum[r] + warp_before(s);
      const bool here = by == 0   ? g >= an && g < an + n
                        : by == 2 ? lane == (int)(g & 31)
                                  : at_sum >= as && at_sum < as + s;
      const uint32_t who = __ballot_sync(0xffffffffu, here);
      const int src = who ? __ffs(who) - 1 : 0;
      b.key = PROBS ? (uint32_t)(0x3fff - (r * 32 + src)) << 16 : logit_key(quick_bits(r, src));
      b.above = __shfl_sync(0xffffffffu, an, src);
      b.count = __shfl_sync(0xffffffffu, n, src);
      b.sum = from_lane(as, src);
      b.w = __shfl_sync(0xffffffffu, w, src);
      return PROBS ? inside(b, by, g, at_sum, key) : b;
    };

    uint32_t keep = total;
    Border last = {0, 0, 0, 0, 0};
    bool cut = false;
    u128 kept_sum = total_sum;
    auto cut_at = [&](uint32_t m, const Border& b) {
      keep = m;
      last = b;
      cut = true;
      kept_sum = b.sum + (u128)b.w * (m - b.above);
    };
    int at = 0;
    float prob = 0.f;
    int edge = 0x7fffffff;
    if (!mark && total > 0) {
      uint32_t k = 0x7fffffffu;
      if (P.top_k && P.top_k[req] > 0) k = (uint32_t)P.top_k[req];
      if (greedy) k = 1;
      if (k < keep && k <= binned) cut_at(k, find(0, k - 1, 0, 0));
      const float top_p = P.top_p && !greedy ? P.top_p[req] : 1.f;
      if (!mark && top_p < 1.f && keep > 1) {
        // the last entry before which less than top_p of the sum lies
        const u128 at = last_place(top_p, kept_sum, total_sum);
        const Border b = find(1, 0, at, 0);
        const uint32_t m = b.above + 1 + quotient(at > b.sum ? at - b.sum : 0, b.w, b.count - 1);
        if (m < keep) cut_at(m, b);
      }
      const float min_p = P.min_p && !greedy ? P.min_p[req] : 0.f;
      if (!mark && min_p > 0.f && keep > 1) {
        uint32_t m = keep;
        if (PROBS) {
          const Border t = find(0, 0, 0, 0);  // the largest
          if (min_p >= 1.f) {
            m = t.count;
          } else if (!mark) {
            const uint32_t key =
                __float_as_uint(__double2float_ru((double)min_p * (double)__uint_as_float(t.key)));
            if (key >> 29 == 1) {
              const Border b = find(2, 0x3fff - (key >> 16), 0, key);
              m = b.above + b.count;
            } else if (far) {
              mark = true;
            }
          }
        } else if (min_p >= 1.f) {
          m = find(0, 0, 0, 0).count;
        } else {
          // the least logit that stays: near an estimate in fp32, 32 of them are weighed (an fp64 logarithm
          // is slow, but right for small shares too)
          const uint32_t topk = logit_key(top_bits);
          uint32_t key;
          if (min_p < kLeastShare) {
            key = min(max(least_logit_key(top_value, T, min_p), 0x80u), topk);
          } else {
            const float unit = fminf(fmaxf(T, 0x1p-100f), 0x1p100f);
            const uint32_t near = orderable(fmaf(unit, __logf(min_p), top_value)) >> 16;
            const uint32_t mine = min(max((int)near - 16 + lane, 1), (int)topk);
            const unsigned long long least_w = __float2ull_rn(min_p * (float)kSumUnit);
            const uint32_t mine_bits = mine & 0x8000u ? mine & 0x7fffu : ~mine & 0xffffu;
            const uint32_t stays = __ballot_sync(0xffffffffu, weight(mine_bits) >= least_w);
            // (the weights ascend with the lane; the estimate is good to a few values, or all is marked)
            const int at0 = stays ? __ffs(stays) - 1 : 32;
            key = __shfl_sync(0xffffffffu, mine, at0 & 31);
            if ((at0 == 0 && near > 16) || (at0 == 32 && near + 16 < topk)) mark = true;
          }
          const uint32_t bits = key & 0x8000u ? key & 0x7fffu : ~key & 0xffffu;
          const uint32_t mag = bits & 0x7fffu;
          if (mag >= 0x4800u) {  // beyond the bins: -2^17 or less (a larger one is not below the top)
            m = far ? (mark = true, keep) : keep;
          } else if (mag < 0x3800u && (mag || smalls)) {
            // between the bins: zero stays or goes
            if (smalls) mark = true;
            else m = bits & 0x8000u ? sh.row_count[129] : sh.row_count[128];
          } else {
            const uint32_t i = mag - 0x3800u;
            const Border b = find(2, mag == 0 ? 128 * 32 : bits & 0x8000u ? 129 * 32 + i : 4095 - i, 0, 0);
            m = b.above + b.count;
          }
        }
        m = max(m, 1u);
        if (!mark && m < keep) cut_at(m, find(0, m - 1, 0, 0));
      }
      if (!mark && !cut && far) {  // all that is a number is kept, or as many as top_k
        if (!PROBS) {
          ask(kOpCount, 0, 0, 0);
          keep = binned + sh.listed;
        }
        if (k < keep) mark = true;
      }
      if (!mark && !WRITE) {
        Border b;
        uint32_t j = 0;
        if (keep == 1) {
          b = cut ? last : find(0, 0, 0, 0);
        } else {
          const u128 at_sum = draw_place(P.u[row], kept_sum, total_sum);
          b = find(1, 0, at_sum, 0);
          j = quotient(at_sum > b.sum ? at_sum - b.sum : 0, b.w, b.count - 1);
          if (!mark && b.above + j >= keep) {
            b = cut ? last : find(0, keep - 1, 0, 0);
            j = keep - 1 - b.above;
          }
        }
        if (!mark) {
          ask(kOpNth, b.key, j, b.count);
          at = sh.index;
          prob = (float)((double)b.w / sum_double(kept_sum));
        }
      }
      if (!mark && WRITE && cut && keep - last.above < last.count) {
        ask(kOpNth, last.key, keep - last.above - 1, last.count);
        edge = sh.index;
      }
    }
    if (lane == 0) {
      sh.edge = edge;
      sh.least = cut ? last.key : 1u;
      if (WRITE) sh.inv = pair_of(kSumUnit / sum_double(kept_sum));
      if (!mark) {
        if (total == 0) raise_err(P.err, SD_ERR_ZERO_ROW);
        if (P.kept) P.kept[row] = (int32_t)keep;
        if (!WRITE) {
          P.tokens[row] = at;
          if (P.prob) P.prob[row] = prob;
        }
      } else if (WRITE) {
        out[0] = kMarkProb;
      } else {
        P.tokens[row] = kMarkToken;
      }
    }
    ask(mark ? kOpMark : total == 0 ? kOpNothing : kOpEnd, 0, 0, 0);
  } else {
    serve();
  }
  if (WRITE) {
    const QuickShared* s0 = cluster.map_shared_rank(&sh, 0);
    const int op = s0->op, edge = s0->edge;
    const uint32_t least = op == kOpNothing ? 0xffffffffu : s0->least;
    if (op != kOpMark) {
      const KeptValue v = {s0->inv, per_unit, top_value, 1.f};
      auto value = [&](int i, uint32_t x) {
        return x < least || (x == least && i > edge) ? 0.f : v.of<PROBS>(x);
      };
      in.write(out, P.vec_out, tid, kQThreads, value);
    }
  }
  meet();  // no CTA leaves while another may read its shared memory
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// ---------------------------------------------------------------------------------------------
// Rows of up to 512 entries (of many rows of probabilities 1024): a warp sorts the row (keys and, upside down, indices, larger first) in
// shared memory and every question is a search in the order itself. Nothing is marked, and no CTA-wide
// barrier is met; bound by the network's instructions. One token of each of 9216 rows of logits, sorted
// against counted: 128 entries 57 us against 350, 700 entries 421 against 400 (of probabilities 424
// against 755), one row of 1000 entries 51 against 28.
// ---------------------------------------------------------------------------------------------
constexpr int kSmallV = 512, kSmallProbsV = 1024, kSmallWarps = 4, kSmallBits = 50;  // sums: multiples of 2^-50

template <bool PROBS, bool WRITE>
__global__ void __launch_bounds__(kSmallWarps * 32, 4) small_rows_kernel(const RowsParams P, int size) {
  extern __shared__ __align__(16) unsigned char s_small[];
  __shared__ float2 s_two_to[64];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (!PROBS) {
    if (threadIdx.x < 64) {
      const double t = exp2((double)threadIdx.x / 64.0);
      const float hi = (float)t;
      s_two_to[threadIdx.x] = make_float2(hi, (float)(t - (double)hi));
    }
    __syncthreads();
  }
  const int row = blockIdx.x * kSmallWarps + warp;
  if (row >= P.n_rows) return;
  const int req = row / P.J, V = P.V;
  const float T = P.temperature ? P.temperature[req] : 1.f;
  const bool greedy = !(T > 0.f);
  unsigned long long* sum = reinterpret_cast<unsigned long long*>(s_small) + warp * 2 * size;
  unsigned long long* item = sum + size;  // key << 32 | ~index
  const RowReader<PROBS> in{P, (const char*)P.rows + (size_t)row * P.ld * (PROBS ? 4 : 2), 0, V};
  for (int i = lane; i < size; i += 32)
    item[i] = i < V ? (unsigned long long)in.key_at(i) << 32 | ~(uint32_t)i : 0ull;
  __syncwarp();
  // a bitonic network: pairs at distance d, larger first in every second run of k
  for (int k = 2; k <= size; k *= 2)
    for (int d = k / 2; d > 0; d /= 2) {
#pragma unroll 4
      for (int t = lane; t < size / 2; t += 32) {
        const int i = (t & -d) * 2 + (t & (d - 1)), j = i + d;
        const unsigned long long a = item[i], b = item[j];
        if ((a < b) == !(i & k)) {
          item[i] = b;
          item[j] = a;
        }
      }
      __syncwarp();
    }
  auto key = [&](int i) { return (uint32_t)(item[i] >> 32); };
  auto index = [&](int i) { return (int)~(uint32_t)item[i]; };
  // how many of the first m have at least this key
  auto at_least = [&](uint32_t k, int m) {
    int lo = 0, hi = m;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (key(mid) >= k) lo = mid + 1;
      else hi = mid;
    }
    return lo;
  };
  const uint32_t top = key(0);
  int live = at_least(1, V);
  if (!PROBS && top == 0xff80u) live = at_least(top, live);  // beside +inf nothing weighs anything
  float* out = WRITE ? P.probs + (size_t)row * P.ld_out : nullptr;
  if (live == 0) {
    if (lane == 0) {
      raise_err(P.err, SD_ERR_ZERO_ROW);
      if (P.kept) P.kept[row] = 0;
      if (!WRITE) {
        P.tokens[row] = 0;
        if (P.prob) P.prob[row] = 0.f;
      }
    }
    if (WRITE)
      for (int i = lane; i < V; i += 32) out[i] = 0.f;
    return;
  }
  const float top_value = PROBS ? 0.f : logit_value(top);
  const int top_exp = PROBS ? max(1, (int)(top >> 23)) : 0;
  float2 per_unit = make_float2(0.f, 0.f);
  if (!PROBS) {
    const double c = 1.4426950408889634074 / fmin(fmax((double)(greedy ? 1.f : T), 0x1p-100), 0x1p100);
    per_unit.x = (float)c;
    per_unit.y = (float)(c - (double)per_unit.x);
  }
  // a logit's weight as a count of 2^-62
  auto weight = [&](uint32_t k) -> unsigned long long {
    if (k == top) return 1ull << kSumBits;
    return weight62(ff_sum(logit_value(k), -top_value), per_unit, s_two_to);
  };
  auto units = [&](uint32_t k) -> unsigned long long {  // of 2^-50
    if (!PROBS) return ((weight(k) >> (kSumBits - 1 - kSmallBits)) + 1) >> 1;
    const unsigned long long sig = (k >> 23 ? 0x800000u : 0u) | (k & 0x7fffffu);
    const int by = max(1, (int)(k >> 23)) - top_exp + kSmallBits - 24;
    return by >= 0 ? sig << by : by < -62 ? 0ull : ((sig >> (-by - 1)) + 1) >> 1;
  };
  // running sums: a lane has a stretch of its own
  const int per = (live + 31) / 32, i0 = min(live, lane * per), i1 = min(live, i0 + per);
  unsigned long long s = 0;
#pragma unroll 2
  for (int i = i0; i < i1; ++i) sum[i] = s += units(key(i));
  const unsigned long long base = warp_before(s);
  for (int i = i0; i < i1; ++i) sum[i] += base;
  __syncwarp();
  // how many of the first m sums are below g (or, equal counted too)
  auto below = [&](unsigned long long g, int m, bool equal) {
    int lo = 0, hi = m;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (sum[mid] < g || (equal && sum[mid] == g)) lo = mid + 1;
      else hi = mid;
    }
    return lo;
  };
  int n = live;
  if (P.top_k && P.top_k[req] > 0) n = min(n, P.top_k[req]);
  if (greedy) n = 1;
  const float top_p = P.top_p && !greedy ? P.top_p[req] : 1.f;
  if (top_p < 1.f && n > 1) {
    const double goal = (double)fmaxf(top_p, 0.f) * (double)sum[n - 1];
    n = min(n, 1 + below((unsigned long long)ceil(goal), n - 1, false));
  }
  const float min_p = P.min_p && !greedy ? P.min_p[req] : 0.f;
  if (min_p > 0.f && n > 1) {
    if (min_p >= 1.f) {
      n = min(n, at_least(top, n));
    } else if (PROBS) {
      const float t = __double2float_ru((double)min_p * (double)__uint_as_float(top));
      n = max(1, at_least(max(1u, __float_as_uint(t)), n));
    } else if (min_p < kLeastShare) {
      n = max(1, at_least(max(1u, least_logit_key(top_value, T, min_p)), n));
    } else {  // 32 places at a time, by their weights
      const double least = (double)min_p * kSumUnit;
      int lo = 0, hi = n;  // the first that goes lies in (lo, hi]; the first of all stays
      while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, at = min(hi - 1, lo + (lane + 1) * step);
        const uint32_t goes = __ballot_sync(0xffffffffu, (double)weight(key(at)) < least);
        const int f = goes ? __ffs(goes) - 1 : 32;
        if (f < 32) hi = min(hi, lo + (f + 1) * step);
        lo = min(hi - 1, lo + f * step);
        if (f == 32) lo = hi - 1;
      }
      n = hi;
    }
  }
  const double kept_sum = (double)sum[n - 1];
  if (lane == 0 && P.kept) P.kept[row] = n;
  if (!WRITE) {
    float u = P.u[row];
    u = u > 0.f ? u : 0.f;
    const double goal = fmin((double)u * kept_sum, kept_sum);
    const int j = min(n - 1, below((unsigned long long)floor(goal), n, true));
    if (lane == 0) {
      P.tokens[row] = index(j);
      if (P.prob) {
        const double w = PROBS ? (double)__uint_as_float(key(j)) : (double)weight(key(j));
        // (in the sums' units: a probability's is 2^-50 of the power of two above the largest)
        const double unit = PROBS ? two_to_the(126 - top_exp + kSmallBits) : two_to_the(kSmallBits - kSumBits);
        P.prob[row] = (float)(w * unit / kept_sum);
      }
    }
  } else {
    const uint32_t least = key(n - 1);
    const int edge = index(n - 1);  // entries of the last value are kept up to here
    const KeptValue v = {pair_of(two_to_the(kSmallBits) / kept_sum), per_unit, top_value,
                         PROBS ? __uint_as_float((uint32_t)(127 + 126 - top_exp) << 23) : 1.f};
    for (int i = lane; i < V; i += 32) {
      const uint32_t x = in.key_at(i);
      // (of entries beside +inf only those that are +inf are kept)
      out[i] = x > least || (x == least && i <= edge)
                   ? !PROBS && x == top ? v.inv.x : v.of<PROBS>(x)
                   : 0.f;
    }
  }
}

template <bool PROBS, bool WRITE>
static int launch_rows(RowsParams& P, cudaStream_t stream) {
  constexpr int kQuickBytes = kQBins * 4 * (PROBS ? 2 : 1);
  static std::atomic<bool> set[kMostDevices];  // true only once the attributes are in force
  int dev = 0;
  const int n_sm = device_sms(dev);
  if (n_sm == 0) return SD_E_DEVICE;
  if (!set[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(rows_kernel<PROBS, WRITE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kHistBytes) != cudaSuccess ||
        cudaFuncSetAttribute(quick_kernel<PROBS, WRITE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kQuickBytes) != cudaSuccess ||
        cudaFuncSetAttribute(small_rows_kernel<PROBS, WRITE>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kSmallWarps * kSmallProbsV * 16) != cudaSuccess)
      return SD_E_LAUNCH;
    set[dev].store(true, std::memory_order_release);
  }
  // (probabilities take the quick kernel longer: with many rows the warps' sorting pays up to 1024)
  if (P.V <= kSmallV || (PROBS && P.V <= kSmallProbsV && P.n_rows >= 4 * n_sm)) {
    int size = 2;
    while (size < P.V) size *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((P.n_rows + kSmallWarps - 1) / kSmallWarps), 1, 1);
    cfg.blockDim = dim3(kSmallWarps * 32, 1, 1);
    cfg.dynamicSmemBytes = (size_t)kSmallWarps * size * 16;
    cfg.stream = stream;
    return cudaLaunchKernelEx(&cfg, small_rows_kernel<PROBS, WRITE>, P, size) == cudaSuccess
               ? SD_OK
               : SD_E_LAUNCH;
  }
  auto parts = [&](int C) { return ((P.V + C - 1) / C + 7) / 8 * 8; };
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = attr;

  // CTAs of a row: more while the SMs have room for them, and a CTA some thousands of entries. Long
  // rows of probabilities are read again for every place that is looked for: with four CTAs a row
  // those on the SMs at a time stay within L2. With 1, 2, 4 CTAs 384 rows of 201088 probabilities cut
  // take 544, 526, 464 us, 2048 of logits 973, 986, 1072, one token of each of 1024 rows 340, 352, 388.
  int C = PROBS && P.V > 65536 ? 4 : 1;
  while (C < kMostClusters && P.n_rows * 2L * C <= 4L * n_sm && P.V > 4096 * C) C *= 2;
  P.part = parts(C);
  attr[0].val.clusterDim.x = (unsigned)C;
  cfg.gridDim = dim3((unsigned)(P.n_rows * C), 1, 1);
  cfg.blockDim = dim3(kQThreads, 1, 1);
  cfg.dynamicSmemBytes = kQuickBytes;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, quick_kernel<PROBS, WRITE>, P) != cudaSuccess) return SD_E_LAUNCH;

  // A part's counts have 16 bits there.
  C = P.V <= 8192 ? 1 : P.V <= 32768 ? 2 : P.V <= 262112 ? 4 : 8;
  P.part = parts(C);
  attr[0].val.clusterDim.x = (unsigned)C;
  const int clusters = n_sm / C < P.n_rows ? n_sm / C : P.n_rows;
  cfg.gridDim = dim3((unsigned)(clusters * C), 1, 1);
  cfg.blockDim = dim3(kRowThreads, 1, 1);
  cfg.dynamicSmemBytes = kHistBytes;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, rows_kernel<PROBS, WRITE>, P) == cudaSuccess ? SD_OK
                                                                              : SD_E_LAUNCH;
}

}  // namespace sdk

extern "C" int sd_rows_launch(int B, int J, int V, int dtype, const void* rows, long ld,
                              const float* temperature, const int32_t* top_k, const float* top_p,
                              const float* min_p, float* probs, long ld_out, const float* u,
                              int32_t* tokens, float* prob, int32_t* kept, int32_t* err,
                              cudaStream_t stream) {
  sdk::RowsParams P;
  const int size = dtype == SD_F32_PROBS ? 4 : 2;
  P.rows = rows;
  P.ld = ld;
  P.J = J;
  P.V = V;
  P.vec = (uintptr_t)rows % 16 == 0 && ld * size % 16 == 0;
  P.temperature = temperature;
  P.top_k = top_k;
  P.top_p = top_p;
  P.min_p = min_p;
  P.probs = probs;
  P.ld_out = ld_out;
  P.vec_out = (uintptr_t)probs % 16 == 0 && ld_out % 4 == 0;
  P.u = u;
  P.tokens = tokens;
  P.prob = prob;
  P.kept = kept;
  P.err = err;
  P.n_rows = B * J;
  if (dtype == SD_F32_PROBS)
    return probs ? sdk::launch_rows<true, true>(P, stream) : sdk::launch_rows<true, false>(P, stream);
  return probs ? sdk::launch_rows<false, true>(P, stream) : sdk::launch_rows<false, false>(P, stream);
}
