// sd_logprobs.cu -- log probabilities of given tokens, with the row's entropy, the token's rank and
// the row's best alternatives (sd_token_logprobs), in one pass over each row.
//
// With y = l / T and m = max y: Z = sum e^(y - m), log p(x) = y_x - m - ln Z, and
// H = -sum p ln p = ln Z - (sum e^(y - m) (y - m)) / Z. Sums are fp32, each thread's own and then a
// tree's. Probability rows need no Z: log p = ln p_x, H = -sum p ln p.
//
// A warp takes 256 neighbouring entries (a group) at a time. The group's maximum, one warp
// reduction, serves twice: as the running maximum of the softmax (it is the same in every lane, so
// a rescale is a branch of the whole warp) and, kept in shared memory, to find the best n entries:
// they lie in the n groups that come first by (maximum, lowest index), because each of those
// holds an entry that beats everything of any later group. Only these n groups are read again.
// Bound by memory: the row once.

#include "sd_common.cuh"

namespace sdk {

constexpr int kLpThreads = 512, kLpWarps = kLpThreads / 32, kGroup = 256;
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
  if (vec && g0 + kGroup <= V) {
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

struct Sums {
  float m, z, s;  // logits: max of l, sum 2^t, sum t 2^t with t = (l - m) c; probabilities: s only
};

// Joins sums over different maxima; c = log2(e) / T.
__device__ __forceinline__ Sums join(const Sums& a, const Sums& b, float c) {
  Sums r;
  r.m = fmaxf(a.m, b.m);
  const float da = a.m == r.m ? 0.f : fmaxf((a.m - r.m) * c, -1e4f);
  const float db = b.m == r.m ? 0.f : fmaxf((b.m - r.m) * c, -1e4f);
  const float fa = ex2(da), fb = ex2(db);
  r.z = a.z * fa + b.z * fb;
  r.s = (a.s + da * a.z) * fa + (b.s + db * b.z) * fb;
  return r;
}

struct LpShared {
  Sums warp_sums[kLpWarps];
  int warp_rank[kLpWarps];
  Sums sums[kLpMaxCluster];     // rank 0's, written by every CTA of the cluster
  int rank[kLpMaxCluster];
  uint64_t best[kLpMaxCluster][SD_TOP_MAX];
  int first[SD_TOP_MAX];        // the groups that hold this CTA's best entries
  int count;
  uint64_t floor;               // no entry below it is among the best
};

template <int DT>
__global__ void __launch_bounds__(kLpThreads) logprob_kernel(const LpParams P) {
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
  const bool in_range = token < P.V;
  float xt = INFINITY;
  if (in_range)
    xt = DT == SD_BF16_LOGITS ? __uint_as_float((uint32_t)((const uint16_t*)x)[token] << 16)
                              : ((const float*)x)[token];
  float T = DT == SD_BF16_LOGITS && P.temperature ? P.temperature[row / P.J] : 1.f;
  if (!(T > 0.f)) T = 1.f;  // a greedy request's rows are reported at temperature 1
  const float inv_T = 1.f / T;
  const float c = kLog2e * inv_T;

  const int begin = part * P.span;
  const int end = min(P.V, begin + P.span);
  const int groups = begin < end ? (end - begin + kGroup - 1) / kGroup : 0;
  float* gmax = reinterpret_cast<float*>(s_dyn);  // [span / kGroup]
  uint64_t* cand = reinterpret_cast<uint64_t*>(s_dyn + ((P.span / kGroup * 4 + 15) & ~15));

  // 1. One pass: sums, rank, group maxima.
  Sums a{-INFINITY, 0.f, 0.f};
  int better = 0;
  constexpr int U = DT == SD_BF16_LOGITS ? 4 : 2;  // groups in flight: 64 bytes a lane
  for (int g = warp; g < groups; g += kLpWarps * U) {
    Raw<DT> raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int gi = g + u * kLpWarps;
      if (gi < groups) raw[u] = load_group<DT>(x, begin + gi * kGroup, P.V, vec, lane);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int gi = g + u * kLpWarps;
      if (gi >= groups) break;
      const int g0 = begin + gi * kGroup;
      float v[8];
      unpack<DT>(raw[u], v);
      float gm = v[0];
#pragma unroll
      for (int e = 1; e < 8; ++e) gm = fmaxf(gm, v[e]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) gm = fmaxf(gm, __shfl_xor_sync(0xffffffffu, gm, o));
      if (lane == 0) gmax[gi] = gm;
      if (DT == SD_BF16_LOGITS) {
        if (gm > a.m) {
          const float d = a.m == -INFINITY ? 0.f : fmaxf((a.m - gm) * c, -1e4f);
          const float f = ex2(d);
          a.s = (a.s + d * a.z) * f;
          a.z *= f;
          a.m = gm;
        }
        if (a.m != -INFINITY) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float t = fmaxf((v[e] - a.m) * c, -1e4f);  // -inf: 2^t is 0, and t 2^t too
            const float p = v[e] == v[e] ? ex2(t) : nanf("");
            a.z += p;
            a.s = fmaf(t, p, a.s);
          }
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) a.s += p_log2_p(v[e]);
      }
      // how many come before the token: larger ones, and equal ones of a lower index
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int i = g0 + entry<DT>(lane, e);
        better += (v[e] > xt || (v[e] == xt && i < token)) && i < P.V;
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Sums b{__shfl_xor_sync(0xffffffffu, a.m, o), __shfl_xor_sync(0xffffffffu, a.z, o),
           __shfl_xor_sync(0xffffffffu, a.s, o)};
    if (DT == SD_BF16_LOGITS) a = join(a, b, c);
    else a.s += b.s;
    better += __shfl_xor_sync(0xffffffffu, better, o);
  }
  if (lane == 0) {
    sm.warp_sums[warp] = a;
    sm.warp_rank[warp] = better;
  }
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
    for (int o = 16; o > 0; o >>= 1) {
      Sums d{__shfl_xor_sync(0xffffffffu, b.m, o), __shfl_xor_sync(0xffffffffu, b.z, o),
             __shfl_xor_sync(0xffffffffu, b.s, o)};
      if (DT == SD_BF16_LOGITS) b = join(b, d, c);
      else b.s += d.s;
      r += __shfl_xor_sync(0xffffffffu, r, o);
    }
    if (lane == 0) {
      root->sums[part] = b;
      root->rank[part] = r;
    }
  } else if (warp == 1 && n > 0) {
    uint64_t mine = 0;  // this lane's best group that is not taken yet
    for (int g = lane; g < groups; g += 32) mine = max(mine, key_of(gmax[g], g) );
    uint64_t last = 0;
    for (int k = 0; k < ng; ++k) {
      uint64_t b = mine;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) b = max(b, __shfl_xor_sync(0xffffffffu, b, o));
      const int g = (int)~(uint32_t)b;
      if (lane == 0) sm.first[k] = g;
      last = b;
      if (mine == b) {  // the next one of this lane
        mine = 0;
        for (int i = lane; i < groups; i += 32) {
          const uint64_t q = key_of(gmax[i], i);
          if (q < b) mine = max(mine, q);
        }
      }
    }
    // with n groups, n entries reach the last one's maximum
    if (lane == 0) sm.floor = ng == n ? (last >> 32) << 32 : 0;
  }
  __syncthreads();

  // 3. The entries of those groups that may be among the best.
  if (n > 0) {
    const uint64_t floor = sm.floor;
    for (int k = warp; k < ng; k += kLpWarps) {
      const int g0 = begin + sm.first[k] * kGroup;
      const Raw<DT> raw = load_group<DT>(x, g0, P.V, vec, lane);
      float v[8];
      unpack<DT>(raw, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int i = g0 + entry<DT>(lane, e);
        const uint64_t q = key_of(v[e], i);
        if (i < P.V && q >= floor) cand[atomicAdd(&sm.count, 1)] = q;
      }
    }
    __syncthreads();
    // their order by counting, which does not depend on the order that they were found in
    const int m = sm.count;
    for (int k = tid; k < m; k += kLpThreads) {
      const uint64_t q = cand[k];
      int before = 0;
      for (int i = 0; i < m; ++i) before += cand[i] > q;
      if (before < n) root->best[part][before] = q;
    }
    for (int k = m + tid; k < n; k += kLpThreads) root->best[part][k] = 0;
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
  const float ln_z = DT == SD_BF16_LOGITS ? logf(t.z) : 0.f;
  auto lp = [&](float v) {
    return DT == SD_BF16_LOGITS ? (v - t.m) * inv_T - ln_z : logf(v);
  };
  if (tid == 0) {
    P.logprob[row] = in_range ? lp(xt) : -INFINITY;
    if (P.entropy)
      P.entropy[row] = DT == SD_BF16_LOGITS ? ln_z - t.s * kLn2 / t.z : 0.f - t.s * kLn2;
    if (P.rank) P.rank[row] = in_range ? rank + 1 : 0;
    if (!in_range) raise_err(P.err, SD_ERR_TOKEN_RANGE);
  }
  if (n > 0) {
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
  // Few rows: a cluster of CTAs shares one, until the rows fill two CTAs on every SM or a CTA has
  // less than 8 groups for each warp pair.
  int C = 1;
  while (C < sdk::kLpMaxCluster && (long)P.rows * C < 2 * 152 && V / (2 * C) >= 4096) C *= 2;
  while (C < sdk::kLpMaxCluster && V / C > SD_TOP_MAX_V / sdk::kLpMaxCluster) C *= 2;
  const long span = ((long)V + C - 1) / C;
  P.span = (int)((span + sdk::kGroup - 1) / sdk::kGroup * sdk::kGroup);
  const size_t smem = (((size_t)P.span / sdk::kGroup * 4 + 15) & ~(size_t)15) +
                      (size_t)n_top * sdk::kGroup * 8;
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
  auto kernel = dtype == SD_BF16_LOGITS ? sdk::logprob_kernel<SD_BF16_LOGITS>
                                        : sdk::logprob_kernel<SD_F32_PROBS>;
  if (smem > 32 * 1024 &&
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
          cudaSuccess)
    return SD_E_LAUNCH;
  return cudaLaunchKernelEx(&cfg, kernel, P) == cudaSuccess ? SD_OK : SD_E_LAUNCH;
}
