// sd_logprobs.cu -- log probabilities of given tokens, with the row's entropy, the token's rank and
// the row's best alternatives (sd_token_logprobs), in one pass over each row.
//
// With y = l / T and m a reference near the largest y: Z = sum e^(y - m), log p(x) = y_x - m - ln Z,
// and H = -sum p ln p = ln Z - (sum e^(y - m) (y - m)) / Z. Sums are fp32, each thread's own and then a
// tree's. Probability rows need no Z: log p = ln p_x, H = -sum p ln p.
//
// A warp takes 256 or 1024 neighbouring entries (a group) at a time. The group's maximum, one warp
// reduction, is kept in shared memory to find the best n entries: they lie in the n groups that
// come first by (maximum, lowest index), because each of those holds an entry that beats everything
// of any later group. Only these n groups are read again (from L2). Entries are compared and
// bounded two at a time as they are stored; only the exponential and the sums take single fp32
// values.
//
// Bound by memory on paper, the row once: 9216 rows of 201088 logits with 20 alternatives, 2.04 GB
// of rows with a token, take 405 us, 74% of the copy rate. The rest goes to instructions: at 16 a clock
// and SM the exponentials alone take 220 us. CTAs of 128 threads, eight on an SM, so that one
// row's tail (the selection, some 3 us) overlaps seven others' loads (434 instead of 396 us with 256
// threads, four on an SM). 5 rows of 1024 probabilities with 5 alternatives: 4.5 us in a graph. 5
// rows of 201088 logits, 2 MB, take 21 us: a row has 8 CTAs at most, a lane one load in flight, and
// the selection up to 20 rounds in a row.

#include "sd_common.cuh"

namespace sdk {

constexpr int kLpThreads = 128, kLpWarps = kLpThreads / 32;
constexpr int kVec = 256;  // entries that a warp loads at once, 8 a lane; a group is U of them
constexpr int kCandidates = 512;
constexpr int kLpMaxCluster = 8;
constexpr float kLn2 = 0.6931471805599453f;

struct LpParams {
  int rows, J, V, n_top, span;  // span: entries of one CTA, a multiple of kGroup
  const void* x;
  long ld;
  const int32_t* tokens;
  const float* temperature;
  float* logprob;
  float* entropy;
  int32_t* rank;
  int32_t* top_ids;
  float* top_lp;
  int32_t* err;
};

// A value's place in an ascending order of 32-bit whole numbers (-0 equal to 0, NaN lowest).
__device__ __forceinline__ uint32_t order_of(float v) {
  if (v != v) return 0;
  const uint32_t b = __float_as_uint(v + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
// Larger is better: the value first, then the lower index.
__device__ __forceinline__ uint64_t key_of(float v, int i) {
  return (uint64_t)order_of(v) << 32 | (uint32_t)~i;
}

// The 8 entries of a lane: 256 entries of a group lie as 32 x 8 (bf16, one 16-byte load a lane) or
// as 2 x 32 x 4 (fp32, two).
template <int DT>
__device__ __forceinline__ int entry(int lane, int e) {
  return DT == SD_BF16_LOGITS ? lane * 8 + e : (e >> 2) * 128 + lane * 4 + (e & 3);
}

template <int DT>
struct Raw {
  uint4 a, b;  // b: fp32 only
};

template <int DT>
__device__ __forceinline__ void unpack(const Raw<DT>& r, float (&v)[8]) {
  const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if (DT == SD_BF16_LOGITS)
      v[e] = e & 1 ? __uint_as_float(w[e >> 1] & 0xffff0000u) : __uint_as_float(w[e >> 1] << 16);
    else
      v[e] = __uint_as_float(w[e]);
  }
}

// Entries past the row's end count as -inf (logits) or 0 (probabilities).
template <int DT>
__device__ __forceinline__ Raw<DT> load_group(const void* row, int g0, int V, bool vec, int lane) {
  Raw<DT> r;
  r.b = make_uint4(0, 0, 0, 0);
  if (vec && g0 + kVec <= V) {
    if (DT == SD_BF16_LOGITS) {
      r.a = __ldg(reinterpret_cast<const uint4*>((const uint16_t*)row + g0) + lane);
    } else {
      const uint4* p = reinterpret_cast<const uint4*>((const float*)row + g0);
      r.a = __ldg(p + lane);
      r.b = __ldg(p + 32 + lane);
    }
    return r;
  }
  uint32_t w[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int i = g0 + entry<DT>(lane, e);
    if (DT == SD_BF16_LOGITS)
      w[e] = i < V ? __ldg((const uint16_t*)row + i) : 0xff80u;
    else
      w[e] = i < V ? __ldg((const uint32_t*)row + i) : 0u;
  }
  if (DT == SD_BF16_LOGITS) {
    r.a = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
  } else {
    r.a = make_uint4(w[0], w[1], w[2], w[3]);
    r.b = make_uint4(w[4], w[5], w[6], w[7]);
  }
  return r;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// p log2 p. The fast logarithm is off by up to 2^-22 absolutely, too much near p = 1 where log2 p
// is small itself; at most one entry of a distribution is above 1/2.
__device__ __forceinline__ float p_log2_p(float p) {
  if (!(p > 0.f)) return p < 0.f || p != p ? nanf("") : 0.f;
  return p * (p > 0.5f ? log2f(p) : __log2f(p));
}

// Logits: a reference logit ref, z = sum 2^t and s = sum t 2^t with t = c l - r, c = log2(e) / T and
// r = ref c rounded once; probabilities: s = sum p log2 p.
struct Sums {
  float ref, z, s;
};

// The temperature of a row: c = log2(e) / T, and what of its logits is taken with it as it stands.
// Where |ref| c passes 2^26, bf16 logits that differ from ref do so by 2^18 units or more, products
// can overflow and r's rounding is no small part of a binade: a row with a logit from `to` on, or
// without one above `from`, is taken by extreme_sums. `low`, 2^27 units below 0, stands for what is
// below it: 2^t is 0 there under any reference, and t 2^t too because t stays finite (-inf would
// make it NaN).
struct Heat {
  float c, from, to;
  __nv_bfloat162 low;
};
__device__ __forceinline__ Heat heat_of(float c) {
  const float most = 67108864.f / c;
  return Heat{c, -most, most, __float2bfloat162_rn(-2.f * most)};
}

// Joins sums over different references (-inf: none yet, +inf: one beyond Heat::to).
__device__ __forceinline__ float shift_of(float from, float to, float c) {
  return from == to ? 0.f : fmaxf(__fmul_rn(from, c) - __fmul_rn(to, c), -1e4f);
}
__device__ __forceinline__ Sums join(const Sums& a, const Sums& b, float c) {
  Sums q;
  q.ref = fmaxf(a.ref, b.ref);
  const float da = shift_of(a.ref, q.ref, c), db = shift_of(b.ref, q.ref, c);
  const float fa = ex2(da), fb = ex2(db);
  q.z = a.z * fa + b.z * fb;
  q.s = (a.s + da * a.z) * fa + (b.s + db * b.z) * fb;
  return q;
}

__device__ __forceinline__ float2 lp_fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(*reinterpret_cast<unsigned long long*>(&d))
      : "l"(*reinterpret_cast<const unsigned long long*>(&a)),
        "l"(*reinterpret_cast<const unsigned long long*>(&b)),
        "l"(*reinterpret_cast<const unsigned long long*>(&c)));
  return d;
}
__device__ __forceinline__ float2 lp_add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(*reinterpret_cast<unsigned long long*>(&d))
      : "l"(*reinterpret_cast<const unsigned long long*>(&a)),
        "l"(*reinterpret_cast<const unsigned long long*>(&b)));
  return d;
}

struct LpShared {
  Sums warp_sums[kLpWarps];
  int warp_rank[kLpWarps];
  float ref[kLpThreads];        // each thread's own
  Sums sums[kLpMaxCluster];     // rank 0's, written by every CTA of the cluster
  int rank[kLpMaxCluster];
  uint64_t best[kLpMaxCluster][SD_TOP_MAX];
  alignas(16) uint64_t cand[kCandidates];  // (before them the threads' maxima, as order_of())
  uint64_t round[2][kLpWarps];
  int first[SD_TOP_MAX];        // the groups that hold this CTA's best entries
  int count;
  uint32_t floor;               // as order_of(): no entry below it is among the best
};

__device__ __forceinline__ uint64_t warp_max64(uint64_t q) {
  const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(q >> 32));
  const uint32_t lo =
      __reduce_max_sync(0xffffffffu, (uint32_t)(q >> 32) == hi ? (uint32_t)q : 0u);
  return (uint64_t)hi << 32 | lo;
}

__device__ __forceinline__ __nv_bfloat162 as_bf162(uint32_t w) {
  return *reinterpret_cast<const __nv_bfloat162*>(&w);
}

// A lane's running sums, in pairs, and how many entries come before the token; t = c l + nr. An entry
// above `edge` moves the reference (kept in LpShared::ref).
struct Lane {
  float edge, nr;
  float2 z, s;
  int better;
};

// Moves a lane's reference up to gm.
__device__ __forceinline__ void move_to(Lane& q, float& ref, float gm, const Heat& heat) {
  if (!(gm < heat.to)) {
    ref = q.edge = INFINITY;
    return;
  }
  const float nr = -__fmul_rn(gm, heat.c);
  const float d = ref == -INFINITY ? -1e4f : fmaxf(nr - q.nr, -1e4f);
  const float f = ex2(d);
  q.s = make_float2((q.s.x + d * q.z.x) * f, (q.s.y + d * q.z.y) * f);
  q.z = make_float2(q.z.x * f, q.z.y * f);
  q.nr = nr;
  ref = gm;
  // it moves only when it is 8 units behind (the sums have room, and a logarithm near 0 still comes from
  // numbers near 0)
  q.edge = fmaf(heat.to, 1.1920929e-7f, gm);  // (2^-23 of 2^26 units)
}

// Sums of a thread's logits of the whole row, whatever they are: the reference is their largest, what is
// below it weighs nothing where it is beyond Heat's range (a step of bf16 is 2^18 units there).
__device__ __noinline__ Sums extreme_sums(const uint16_t* x, int V, const Heat& heat) {
  Sums q{-INFINITY, 0.f, 0.f};
  for (int i = threadIdx.x; i < V; i += kLpThreads) {
    const float v = __uint_as_float((uint32_t)__ldg(x + i) << 16);
    if (v != v || v == INFINITY) q.z = nanf("");
    if (!(v > -INFINITY) || v == INFINITY) continue;
    if (v > q.ref) {
      const float d = shift_of(q.ref, v, heat.c), f = ex2(d);
      q.s = (q.s + d * q.z) * f;
      q.z *= f;
      q.ref = v;
    }
    if (fabsf(q.ref) < heat.to) {
      const float t = fmaxf(fmaf(v, heat.c, -__fmul_rn(q.ref, heat.c)), -1e4f), p = ex2(t);
      q.z += p;
      q.s += t * p;
    } else if (v == q.ref) {
      q.z += 1.f;
    }
  }
  return q;
}

// Takes in a group of U vectors a lane (entries g0 .. g0 + 256 U - 1); returns the lane's largest.
template <int DT, int U>
__device__ __forceinline__ float take(Lane& q, const Raw<DT> (&raw)[U], const Heat& heat,
                                      float& ref, float xt, int g0, int token, int V, int lane) {
  float gm;
  // a group that holds the token or ends the row is looked at entry by entry for the rank
  const bool edge = (token >= g0 && token < g0 + U * kVec) || g0 + U * kVec > V;
  if (DT == SD_BF16_LOGITS) {
    __nv_bfloat162 m2 = as_bf162(raw[0].a.x);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const __nv_bfloat162 h = __hmax2(__hmax2(as_bf162(raw[u].a.x), as_bf162(raw[u].a.y)),
                                       __hmax2(as_bf162(raw[u].a.z), as_bf162(raw[u].a.w)));
      m2 = u == 0 ? h : __hmax2(m2, h);
    }
    gm = fmaxf(__low2float(m2), __high2float(m2));
    if (!edge && !(gm < xt)) {
      // entries before the token count from equality on, those behind it from above it on
      const __nv_bfloat162 x2 = __float2bfloat162_rn(xt);
      __nv_bfloat162 n2 = __float2bfloat162_rn(0.f);
      if (g0 < token) {
#pragma unroll
        for (int u = 0; u < U; ++u)
          n2 = __hadd2(n2, __hadd2(__hadd2(__hge2(as_bf162(raw[u].a.x), x2),
                                           __hge2(as_bf162(raw[u].a.y), x2)),
                                   __hadd2(__hge2(as_bf162(raw[u].a.z), x2),
                                           __hge2(as_bf162(raw[u].a.w), x2))));
      } else {
#pragma unroll
        for (int u = 0; u < U; ++u)
          n2 = __hadd2(n2, __hadd2(__hadd2(__hgt2(as_bf162(raw[u].a.x), x2),
                                           __hgt2(as_bf162(raw[u].a.y), x2)),
                                   __hadd2(__hgt2(as_bf162(raw[u].a.z), x2),
                                           __hgt2(as_bf162(raw[u].a.w), x2))));
      }
      q.better += (int)(__low2float(n2) + __high2float(n2));
    }
    if (gm > q.edge) move_to(q, ref, gm, heat);
    // (NaN stays)
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t w[4] = {raw[u].a.x, raw[u].a.y, raw[u].a.z, raw[u].a.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = __bfloat1622float2(__hmax2_nan(as_bf162(w[i]), heat.low));
        const float2 t = lp_fma2(f, make_float2(heat.c, heat.c), make_float2(q.nr, q.nr));
        const float2 p = make_float2(ex2(t.x), ex2(t.y));
        q.z = lp_add2(q.z, p);
        q.s = lp_fma2(t, p, q.s);
      }
    }
  } else {
    gm = -INFINITY;
    int n = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float v[8];
      unpack<DT>(raw[u], v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        gm = fmaxf(gm, v[e]);
        n += g0 < token ? v[e] >= xt : v[e] > xt;
      }
#pragma unroll
      for (int e = 0; e < 8; e += 2)
        q.s = lp_add2(q.s, make_float2(p_log2_p(v[e]), p_log2_p(v[e + 1])));
    }
    if (!edge) q.better += n;
  }
  if (edge) {
    int n = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float v[8];
      unpack<DT>(raw[u], v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int i = g0 + u * kVec + entry<DT>(lane, e);
        n += (v[e] > xt || (v[e] == xt && i < token)) && i < V;
      }
    }
    q.better += n;
  }
  return gm;
}

// More entries reach the floor than there is room for: those above it, and the first of those at it.
// Their number, 0 if those above it are too many as well. Out of line, so that it does not weigh on
// the pass over the row (9216 rows of 201088 logits: 407 us with it inside, 404 without).
template <int DT, int U>
__device__ __noinline__ int of_many(LpShared& sm, const void* x, int begin, int V, bool vec, int ng,
                                    int n) {
  constexpr int kGroup = U * kVec;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t floor = sm.floor;
  const float least = value_of(floor), bound = value_of(floor + 1);
  __syncthreads();
  if (threadIdx.x == 0) sm.count = 0;
  __syncthreads();
  for (int k = warp; k < ng * U; k += kLpWarps) {
    const int g0 = begin + sm.first[k / U] * kGroup + (k % U) * kVec;
    const Raw<DT> r = load_group<DT>(x, g0, V, vec, lane);
    float v[8];
    unpack<DT>(r, v);
    int full = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int i = g0 + entry<DT>(lane, e);
      if (v[e] >= bound && i < V) {
        const int at = atomicAdd(&sm.count, 1);
        if (at < kCandidates) sm.cand[at] = key_of(v[e], i);
        else full = 1;
      }
    }
    if (full) break;
  }
  __syncthreads();
  const int m = sm.count;
  if (m > kCandidates) return 0;
  if (m >= n) return m;
  __syncthreads();
  if (warp == 0) {  // the groups in the order of their indices
    const int f = lane < ng ? sm.first[lane] : 0x7fffffff;
    int place = 0;
    for (int i = 0; i < ng; ++i) place += __shfl_sync(0xffffffffu, f, i) < f;
    if (lane < ng) sm.first[place] = f;
    __syncwarp();
    int to = m;
    for (int k = 0; to < n && k < ng * U; ++k) {
      const int g0 = begin + sm.first[k / U] * kGroup + (k % U) * kVec;
      const Raw<DT> r = load_group<DT>(x, g0, V, vec, lane);
      float v[8];
      unpack<DT>(r, v);
      constexpr int kRun = DT == SD_BF16_LOGITS ? 8 : 4;  // a lane's neighbouring entries
#pragma unroll
      for (int e0 = 0; e0 < 8; e0 += kRun) {
        int mine = 0;
#pragma unroll
        for (int e = e0; e < e0 + kRun; ++e)
          mine += v[e] == least && g0 + entry<DT>(lane, e) < V;
        int upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += y;
        }
        int at = to + upto - mine;
#pragma unroll
        for (int e = e0; e < e0 + kRun; ++e) {
          const int i = g0 + entry<DT>(lane, e);
          if (v[e] == least && i < V) {
            if (at < n) sm.cand[at] = key_of(v[e], i);
            ++at;
          }
        }
        to += __shfl_sync(0xffffffffu, upto, 31);
      }
    }
    if (lane == 0) sm.count = min(to, n);
  }
  __syncthreads();
  return sm.count;
}

template <int DT, int U>
__global__ void __launch_bounds__(kLpThreads, 8) logprob_kernel(const LpParams P) {
  constexpr int kGroup = U * kVec;
  extern __shared__ __align__(16) unsigned char s_dyn[];
  __shared__ LpShared sm;
  const cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), part = (int)cluster.block_rank();
  const int row = blockIdx.x / C;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int token = P.tokens[row];

  if (token < 0) {  // no token here: nothing is read
    if (part == 0) {
      if (tid == 0) {
        P.logprob[row] = 0.f;
        if (P.entropy) P.entropy[row] = 0.f;
        if (P.rank) P.rank[row] = 0;
        if (token != -1) raise_err(P.err, SD_ERR_TOKEN_RANGE);
      }
      if (tid < P.n_top) {
        P.top_ids[(long)row * P.n_top + tid] = -1;
        P.top_lp[(long)row * P.n_top + tid] = -INFINITY;
      }
    }
    return;
  }

  if (C > 1) cluster.barrier_arrive();  // every CTA runs before another writes to its memory
  const int esize = DT == SD_BF16_LOGITS ? 2 : 4;
  const void* x = (const unsigned char*)P.x + (long)row * P.ld * esize;
  const bool vec = (uintptr_t)x % 16 == 0;
  const int begin = part * P.span;
  const int end = min(P.V, begin + P.span);
  const int groups = begin < end ? (end - begin + kGroup - 1) / kGroup : 0;
  uint32_t* gmax = reinterpret_cast<uint32_t*>(s_dyn);  // [span / kGroup], as order_of()

  // 1. One pass: sums, rank, group maxima; the next group on its way while one is taken in.
  Raw<DT> raw[U];
  auto fetch = [&](int g) {
    if (g < groups) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        raw[u] = load_group<DT>(x, begin + g * kGroup + u * kVec, P.V, vec, lane);
    }
  };
  fetch(warp);
  const bool in_range = token < P.V;
  float xt = INFINITY;
  if (in_range)
    xt = DT == SD_BF16_LOGITS ? __uint_as_float((uint32_t)((const uint16_t*)x)[token] << 16)
                              : ((const float*)x)[token];
  float T = DT == SD_BF16_LOGITS && P.temperature ? P.temperature[row / P.J] : 1.f;
  if (!(T > 0.f)) T = 1.f;  // a greedy request's rows are reported at temperature 1
  T = fminf(fmaxf(T, 7.8886090522101181e-31f), 1.2676506002282294e30f);  // 2^-100, 2^100
  const float c = kLog2e / T;
  const Heat heat = heat_of(c);
  sm.ref[tid] = -INFINITY;
  Lane q{heat.from, 0.f, make_float2(0.f, 0.f), make_float2(0.f, 0.f), 0};
  float tm = nanf("");  // the largest entry of this thread
  for (int g = warp; g < groups; g += kLpWarps) {
    Raw<DT> now[U];
#pragma unroll
    for (int u = 0; u < U; ++u) now[u] = raw[u];
    fetch(g + kLpWarps);
    const float gm = take<DT, U>(q, now, heat, sm.ref[tid], xt, begin + g * kGroup, token, P.V, lane);
    if (U == 1) tm = fmaxf(tm, gm);
    if (P.n_top > 0) {
      const uint32_t o = __reduce_max_sync(0xffffffffu, order_of(gm));
      if (lane == 0) gmax[g] = o;
    }
  }
  Sums a{sm.ref[tid], q.z.x + q.z.y, q.s.x + q.s.y};
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Sums b{__shfl_xor_sync(0xffffffffu, a.ref, o), __shfl_xor_sync(0xffffffffu, a.z, o),
           __shfl_xor_sync(0xffffffffu, a.s, o)};
    if (DT == SD_BF16_LOGITS) a = join(a, b, c);
    else a.s += b.s;
  }
  const int rank_part = __reduce_add_sync(0xffffffffu, q.better);
  if (lane == 0) {
    sm.warp_sums[warp] = a;
    sm.warp_rank[warp] = rank_part;
  }
  uint32_t* thread_max = reinterpret_cast<uint32_t*>(sm.cand);
  if (U == 1) thread_max[tid] = order_of(tm);
  if (tid == 0) sm.count = 0;
  if (C > 1) cluster.barrier_wait();
  __syncthreads();

  // 2. Warp 1 finds the first n groups while warp 0 joins the sums.
  LpShared* root = C > 1 ? cluster.map_shared_rank(&sm, 0) : &sm;
  const int n = P.n_top;
  const int ng = min(n, groups);
  if (warp == 0) {
    Sums b = lane < kLpWarps ? sm.warp_sums[lane] : Sums{-INFINITY, 0.f, 0.f};
    int r = lane < kLpWarps ? sm.warp_rank[lane] : 0;
#pragma unroll
    for (int o = kLpWarps / 2; o > 0; o >>= 1) {
      Sums d{__shfl_xor_sync(0xffffffffu, b.ref, o), __shfl_xor_sync(0xffffffffu, b.z, o),
             __shfl_xor_sync(0xffffffffu, b.s, o)};
      if (DT == SD_BF16_LOGITS) b = join(b, d, c);
      else b.s += d.s;
    }
    r = __reduce_add_sync(0xffffffffu, r);
    if (lane == 0) {
      root->sums[part] = b;
      root->rank[part] = r;
    }
  } else if (warp == 1 && groups > n) {
    // lane i watches over groups i, i + 32, ...: key (maximum, lower index first)
    uint64_t mine = 0;
    for (int g = lane; g < groups; g += 32) mine = max(mine, (uint64_t)gmax[g] << 32 | (uint32_t)~g);
    uint64_t best = 0;
    for (int k = 0; k < n; ++k) {
      best = warp_max64(mine);
      const int g = (int)~(uint32_t)best;
      if (lane == 0) sm.first[k] = g;
      // the watcher's next one, looked up by the whole warp
      uint64_t next = 0;
      for (int i = (g & 31) + 32 * lane; i < groups; i += 1024) {
        const uint64_t q = (uint64_t)gmax[i] << 32 | (uint32_t)~i;
        if (q < best) next = max(next, q);
      }
      next = warp_max64(next);
      if (lane == (g & 31)) mine = next;
    }
    if (lane == 0) sm.floor = (uint32_t)(best >> 32);  // n entries reach the last group's maximum
  }
  if (U == 1 && n > 0 && groups <= n) {
    // Every group. The threads hold 128 disjoint parts of the entries: n entries reach the n-th
    // largest of their maxima. (With groups of several vectors a CTA has 57 groups at the least.)
    if (tid < ng) sm.first[tid] = tid;
    const uint32_t mine = thread_max[tid];
    int before = 0;
#pragma unroll 8
    for (int i = 0; i < kLpThreads; i += 4) {
      const uint4 o = *reinterpret_cast<const uint4*>(thread_max + i);
      const uint32_t w[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) before += w[k] > mine || (w[k] == mine && i + k < tid);
    }
    if (before == n - 1) sm.floor = mine;
  }
  __syncthreads();

  // 3. Their entries that reach the floor: few, but for ties (a row that is 0 or -inf but for a
  // few). Then those above the floor, and the first of those at it.
  if (n > 0) {
    const uint32_t floor = sm.floor;
    bool many = floor == 0;
    int m = 0;
    if (!many) {
      const float least = value_of(floor);
      for (int k = warp; k < ng * U; k += kLpWarps) {
        const int g0 = begin + sm.first[k / U] * kGroup + (k % U) * kVec;
        const Raw<DT> r = load_group<DT>(x, g0, P.V, vec, lane);
        float v[8];
        unpack<DT>(r, v);
        int full = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int i = g0 + entry<DT>(lane, e);
          if (v[e] >= least && i < P.V) {
            const int at = atomicAdd(&sm.count, 1);
            if (at < kCandidates) sm.cand[at] = key_of(v[e], i);
            else full = 1;
          }
        }
        if (full) break;  // (rows cut to 9 entries 525 us without, full ones 404 us instead of 401)
      }
      __syncthreads();
      m = sm.count;
      if (m > kCandidates)
        m = of_many<DT, U>(sm, x, begin, P.V, vec, ng, n);
      many = m < n;  // (what lies past the row's end was among the maxima)
    }
    if (!many) {
      // their order by counting, which does not depend on the order that they were found in
      for (int k = tid; k < m; k += kLpThreads) {
        const uint64_t q = sm.cand[k];
        int before = 0;
        for (int i = 0; i < m; ++i) before += sm.cand[i] > q;
        if (before < n) root->best[part][before] = q;
      }
    } else {
      // fewer than n numbers here, or hundreds above the floor: n rounds, each thread with its best
      // one not yet taken
      const int items = ng * kGroup;
      auto best_below = [&](uint64_t limit) {
        uint64_t b = 0;
        for (int k = tid; k < items; k += kLpThreads) {
          const int i = begin + sm.first[k / kGroup] * kGroup + k % kGroup;
          if (i >= P.V) continue;
          const float v = DT == SD_BF16_LOGITS
                              ? __uint_as_float((uint32_t)__ldg((const uint16_t*)x + i) << 16)
                              : __ldg((const float*)x + i);
          const uint64_t q = key_of(v, i);
          if (q < limit) b = max(b, q);
        }
        return b;
      };
      uint64_t mine = best_below(~0ull);
      for (int k = 0; k < n; ++k) {
        const uint64_t w = warp_max64(mine);
        if (lane == 0) sm.round[k & 1][warp] = w;
        __syncthreads();
        uint64_t best = 0;
#pragma unroll
        for (int i = 0; i < kLpWarps; ++i) best = max(best, sm.round[k & 1][i]);
        if (tid == 0) root->best[part][k] = best;
        if (best && mine == best) mine = best_below(best);
      }
    }
  }
  if (C > 1) cluster.sync();
  else __syncthreads();
  if (part != 0) return;

  // 4. The row's answers.
  Sums t = sm.sums[0];
  int rank = sm.rank[0];
  for (int i = 1; i < C; ++i) {
    if (DT == SD_BF16_LOGITS) t = join(t, sm.sums[i], c);
    else t.s += sm.sums[i].s;
    rank += sm.rank[i];
  }
  if (DT == SD_BF16_LOGITS && isinf(t.ref)) {
    t = extreme_sums((const uint16_t*)x, P.V, heat);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      t = join(t, Sums{__shfl_xor_sync(0xffffffffu, t.ref, o), __shfl_xor_sync(0xffffffffu, t.z, o),
                       __shfl_xor_sync(0xffffffffu, t.s, o)}, c);
    __syncthreads();
    if (lane == 0) sm.warp_sums[warp] = t;
    __syncthreads();
    t = sm.warp_sums[0];
    for (int i = 1; i < kLpWarps; ++i) t = join(t, sm.warp_sums[i], c);
  }
  const float log2_z = DT == SD_BF16_LOGITS ? log2f(t.z) : 0.f;
  // z is in units of 2^r, r a rounded ref c: the rest of that comes off
  const float ln_z =
      (log2_z - (fabsf(t.ref) < heat.to ? fmaf(t.ref, c, -__fmul_rn(t.ref, c)) : 0.f)) * kLn2;
  auto lp = [&](float v) { return DT == SD_BF16_LOGITS ? (v - t.ref) * (c * kLn2) - ln_z : logf(v); };
  if (tid == 0) {
    P.logprob[row] = in_range ? lp(xt) : -INFINITY;
    if (P.entropy)
      P.entropy[row] = DT == SD_BF16_LOGITS ? (log2_z - t.s / t.z) * kLn2 : 0.f - t.s * kLn2;
    if (P.rank) P.rank[row] = in_range ? rank + 1 : 0;
    if (!in_range) raise_err(P.err, SD_ERR_TOKEN_RANGE);
  }
  if (C == 1) {  // already in order
    if (tid < n) {
      const uint64_t q = sm.best[0][tid];
      P.top_ids[(long)row * n + tid] = (int32_t)~(uint32_t)q;
      P.top_lp[(long)row * n + tid] = lp(value_of((uint32_t)(q >> 32)));
    }
  } else if (n > 0) {
    for (int k = tid; k < C * n; k += kLpThreads) {
      const uint64_t q = sm.best[k / n][k % n];
      int before = 0;
      for (int i = 0; i < C; ++i)
        for (int j = 0; j < n; ++j) before += sm.best[i][j] > q;
      if (q && before < n) {
        P.top_ids[(long)row * n + before] = (int32_t)~(uint32_t)q;
        P.top_lp[(long)row * n + before] = lp(value_of((uint32_t)(q >> 32)));
      }
    }
  }
}

}  // namespace sdk

extern "C" int sd_logprobs_launch(int B, int J, int V, int dtype, const void* rows, long ld,
                                  const int32_t* tokens, const float* temperature, int n_top,
                                  float* logprob, float* entropy, int32_t* rank, int32_t* top_ids,
                                  float* top_lp, int32_t* err, cudaStream_t stream) {
  sdk::LpParams P;
  P.rows = B * J;
  P.J = J;
  P.V = V;
  P.n_top = n_top;
  P.x = rows;
  P.ld = ld;
  P.tokens = tokens;
  P.temperature = temperature;
  P.logprob = logprob;
  P.entropy = entropy;
  P.rank = rank;
  P.top_ids = top_ids;
  P.top_lp = top_lp;
  P.err = err;
  // Few rows: a cluster of CTAs shares one, until the rows fill eight CTAs on every SM or a CTA has
  // few entries left, while there is a free SM for each fewer. Measured in us, 20 alternatives, 1, 2,
  // 4 or 8 CTAs: 5 rows of 1024 logits 5.7, 7.0, 7.2, 10.8; of 8192 12.7, 9.3, 8.2, 10.6; of 32000
  // 17.7, 15.9, 14.6, 12.6; of 201088 43, 32, 23, 21. 192 rows of 32000: 20.9, 17.5, 17.9, 21.2.
  // 768 rows of 201088: 81, 72, 79, 109. 2304 rows of 131072: 104, 120, 158, 233.
  int C = 1;
  while (C < sdk::kLpMaxCluster && (long)P.rows * C < 8 * 152 &&
         V / (2 * C) >= ((long)P.rows * 2 * C <= 152 ? 2048 : 4096))
    C *= 2;
  while (C < sdk::kLpMaxCluster && V / C > SD_TOP_MAX_V / sdk::kLpMaxCluster) C *= 2;
  // Groups of one vector while there are few of them, so that the best n groups are few entries;
  // of logits else of four, which saves most of a group's own work. One against four vectors: 5
  // rows of 201088 in CTAs of 25136 logits 21 to 26 us, 192 rows in CTAs of 50272 34.6 to 34.8, 2304
  // rows of 131072 in CTAs of 65536 141 to 120, of 131072 152 to 104. Probabilities, which bring half
  // as many entries with each byte, gain nothing (2304 rows of 131072: 222 to 222 us with two).
  const int U = dtype == SD_BF16_LOGITS && V / C >= 65536 ? 4 : 1;
  const int group = U * sdk::kVec;
  const long span = ((long)V + C - 1) / C;
  P.span = (int)((span + group - 1) / group * group);
  const size_t smem = (size_t)P.span / group * 4;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(P.rows * C), 1, 1);
  cfg.blockDim = dim3(sdk::kLpThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto kernel = U > 1                     ? sdk::logprob_kernel<SD_BF16_LOGITS, 4>
                : dtype == SD_BF16_LOGITS ? sdk::logprob_kernel<SD_BF16_LOGITS, 1>
                                          : sdk::logprob_kernel<SD_F32_PROBS, 1>;
  if (smem > 16 * 1024 &&
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
          cudaSuccess)
    return SD_E_LAUNCH;
  return cudaLaunchKernelEx(&cfg, kernel, P) == cudaSuccess ? SD_OK : SD_E_LAUNCH;
}
