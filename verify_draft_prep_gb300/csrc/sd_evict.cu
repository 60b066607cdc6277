// sd_evict.cu -- a cache cut to a budget of tokens a request (sd_kv_evict): which tokens stay, by the
// weight that attention has given them, and their move to the front.
//
// Of a request's tokens the first `sink` and the last `recent` stay, and of those between them the
// ones with the largest weights, equal ones in their order, until there are `budget`. Every KV head
// chooses for itself: the heads of a page need not hold the same tokens, only the same number. What
// stays keeps its order; it fills new pages (or the request's own from the first on).

#include <atomic>

#include "sd_kv.cuh"

namespace sdk {

struct EvictParams {
  KvCache c;
  float* k_scale;
  float* v_scale;
  uint8_t* k;
  uint8_t* v;
  float* weights;  // [num_blocks][Hkv][block_size]
  int B, max_blocks, to_blocks, budget, sink, recent, in_smem;
  const int32_t* table;
  const int32_t* to;  // the new pages; NULL: the request's own
  const int32_t* ctx;
  int32_t* kept;      // [B][Hkv][budget]
  int32_t* new_lens;
  int32_t* err;
};

constexpr int kSelThreads = 512, kSelWarps = kSelThreads / 32;

// Tokens that a request's table covers.
__device__ __forceinline__ long evict_covered(const EvictParams& P) {
  return min((long)P.max_blocks << P.c.log2_bs, 2147483647L - 1023);
}
__device__ __forceinline__ int evict_len(const EvictParams& P, int r) {
  const int n = P.ctx[r];
  return n < 0 ? 0 : (int)min((long)n, evict_covered(P));
}

// ---------------------------------------------------------------------------------------------
// Choice: one CTA a request and head. The weights become orderable keys in shared memory (where they
// fit, 200 KB; else they are read again), three passes of 11, 11 and 10 bits find the last key that
// stays, and a pass in the tokens' order writes down the places.
// ---------------------------------------------------------------------------------------------
__global__ void __launch_bounds__(kSelThreads) evict_choose_kernel(const EvictParams P) {
  extern __shared__ uint32_t s_key[];
  __shared__ uint32_t s_bin[2048];
  __shared__ uint32_t s_warp[kSelWarps], s_warp2[kSelWarps];
  __shared__ uint32_t s_found[2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = blockIdx.x, r = blockIdx.y;
  const int n = evict_len(P, r), ctx = P.ctx[r];
  const int keep = min(n, P.budget);
  int32_t* kept = P.kept + ((long)r * P.c.Hkv + h) * P.budget;
  if (tid == 0 && h == 0) {
    P.new_lens[r] = keep;
    if (ctx < 0 || ctx > evict_covered(P)) raise_err(P.err, SD_ERR_KV_RANGE);
  }
  for (int i = keep + tid; i < P.budget; i += kSelThreads) kept[i] = -1;
  if (n <= P.budget) {
    for (int i = tid; i < n; i += kSelThreads) kept[i] = i;
    return;
  }
  const int32_t* table = P.table + (long)r * P.max_blocks;
  const int bs = 1 << P.c.log2_bs, first = P.sink, m = n - P.sink - P.recent;
  bool bad = false;
  // A token's weight as a key: larger ones first, a NaN before all; one without a page counts as 0.
  auto load = [&](int i) -> uint32_t {
    const int t = first + i;
    const int page = __ldg(table + (t >> P.c.log2_bs));
    if ((unsigned)page >= (unsigned)P.c.num_blocks) {
      bad = true;
      return orderable(0.f);
    }
    const float w = P.weights[((long)page * P.c.Hkv + h) * bs + (t & (bs - 1))];
    return w != w ? 0xffffffffu : orderable(w);
  };
  const bool held = P.in_smem >= m;
  if (held) {
#pragma unroll 8
    for (int i = tid; i < m; i += kSelThreads) s_key[i] = load(i);
  }
  auto key = [&](int i) { return held ? s_key[i] : load(i); };

  uint32_t need = (uint32_t)(P.budget - P.sink - P.recent);  // < m
  uint32_t prefix = 0;
  bool any = need > 0;
  for (int level = 0; any && level < 3; ++level) {
    const int shift = level == 0 ? 21 : level == 1 ? 10 : 0, bits = level == 2 ? 10 : 11;
    const uint32_t high = level == 0 ? 0u : 0xffffffffu << (shift + bits);
    for (int i = tid; i < 2048; i += kSelThreads) s_bin[i] = 0;
    __syncthreads();
    for (int i = tid; i < m; i += kSelThreads) {
      const uint32_t k = key(i);
      if ((k & high) == prefix) atomicAdd(&s_bin[2047 - ((k >> shift) & ((1u << bits) - 1))], 1u);
    }
    __syncthreads();
    // the bin in which number `need` from the largest lies: 4 bins a thread
    uint32_t c[4], sum = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) sum += c[j] = s_bin[tid * 4 + j];
    uint32_t at = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, at, o);
      if (lane >= o) at += x;
    }
    if (lane == 31) s_warp[warp] = at;
    __syncthreads();
    at -= sum;
    for (int w = 0; w < warp; ++w) at += s_warp[w];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (at < need && need <= at + c[j]) {
        s_found[0] = 2047 - (tid * 4 + j);
        s_found[1] = at;
      }
      at += c[j];
    }
    __syncthreads();
    prefix |= s_found[0] << shift;
    need -= s_found[1];
    __syncthreads();
  }
  const uint32_t ties = need;  // of the tokens whose key is `prefix`, so many stay: the first

  // the places, in order: a warp goes over a stretch of its own
  const int seg = (n + kSelWarps * 32 - 1) / (kSelWarps * 32) * 32;
  const int a = min(n, warp * seg), b = min(n, a + seg);
  // 0: goes, 1: stays, 2: stays if it is among the first `ties` of its key
  auto kind = [&](int t) {
    if (t < P.sink || t >= n - P.recent) return 1;
    if (!any) return 0;
    const uint32_t k = key(t - first);
    return k > prefix ? 1 : k == prefix ? 2 : 0;
  };
  uint32_t stay = 0, tied = 0;
  for (int i = a; i < b; i += 32) {
    const int x = i + lane < b ? kind(i + lane) : 0;
    stay += __popc(__ballot_sync(0xffffffffu, x == 1));
    tied += __popc(__ballot_sync(0xffffffffu, x == 2));
  }
  if (lane == 0) {
    s_warp[warp] = stay;
    s_warp2[warp] = tied;
  }
  __syncthreads();
  stay = tied = 0;
  for (int w = 0; w < warp; ++w) {
    stay += s_warp[w];
    tied += s_warp2[w];
  }
  const uint32_t below = (1u << lane) - 1;
  for (int i = a; i < b; i += 32) {
    const int x = i + lane < b ? kind(i + lane) : 0;
    const uint32_t one = __ballot_sync(0xffffffffu, x == 1), two = __ballot_sync(0xffffffffu, x == 2);
    const uint32_t mine = tied + __popc(two & below);
    if (x == 1 || (x == 2 && mine < ties))
      kept[stay + __popc(one & below) + min(mine, ties)] = i + lane;
    stay += __popc(one);
    tied += __popc(two);
  }
  if (bad) raise_err(P.err, SD_ERR_KV_RANGE);
}

// ---------------------------------------------------------------------------------------------
// Move: a CTA takes 128 places (whole pages) of one head, K and V together, into registers and then
// to their new pages. A new page's scale is the largest of its tokens' (their sources' pages'), so that
// values only ever lose what becomes subnormal, and a page of tokens that do not move stays as it is.
// Within the request's own pages a token only moves towards the front: a cluster goes over the
// places in rounds, and nothing is written before all of the round's tokens are read.
// ---------------------------------------------------------------------------------------------
constexpr int kMoveThreads = 256, kMoveTokens = 128, kMoveCluster = 8;

template <bool IN_PLACE>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictParams P) {
  __shared__ long s_src[kMoveTokens], s_dst[kMoveTokens];  // elements; -1: no page, -2: no token
  __shared__ float s_scale[2][kMoveTokens];
  __shared__ unsigned s_max[2][kMoveTokens];  // of each page, in its first token's place
  __shared__ float s_ratio[2][kMoveTokens];   // -1: stays as it is
  const KvCache& c = P.c;
  const int tid = threadIdx.x, h = blockIdx.y, r = blockIdx.z;
  const int n = min(evict_len(P, r), P.budget), bs = 1 << c.log2_bs;
  const int32_t* kept = P.kept + ((long)r * c.Hkv + h) * P.budget;
  const int32_t* table = P.table + (long)r * P.max_blocks;
  const int32_t* to = IN_PLACE ? table : P.to + (long)r * P.to_blocks;
  const int to_blocks = IN_PLACE ? P.max_blocks : P.to_blocks;
  const int parts = c.D / 16;  // 16-byte parts of a token's head
  const int step = IN_PLACE ? kMoveCluster * kMoveTokens : 0x7fffffff;
  for (long j0 = 0; j0 < n; j0 += step) {
    const long base = j0 + (long)blockIdx.x * kMoveTokens;
    // 1. where the tokens come from and go to, and the scales
    float weight = 0.f;
    long weight_to = -1, scale_to = -1;
    if (tid < kMoveTokens) {
      const long j = base + tid;
      long src = -2, dst = -2;
      float sk = 0.f, sv = 0.f;
      s_max[0][tid] = s_max[1][tid] = 0;
      if (j < n) {
        const int t = kept[j];
        const int page = t >= 0 ? table[t >> c.log2_bs] : -1;
        const long b = j >> c.log2_bs;
        const int new_page = b < to_blocks ? to[b] : -1;
        src = dst = -1;
        if ((unsigned)page < (unsigned)c.num_blocks) {
          const int off = t & (bs - 1);
          src = page * c.st_block + off * c.st_tok + h * c.st_head;
          sk = P.k_scale[(long)page * c.Hkv + h];
          sv = P.v_scale[(long)page * c.Hkv + h];
          weight = P.weights[((long)page * c.Hkv + h) * bs + off];
        }
        if ((unsigned)new_page < (unsigned)c.num_blocks) {
          const int off = (int)(j & (bs - 1));
          dst = new_page * c.st_block + off * c.st_tok + h * c.st_head;
          weight_to = ((long)new_page * c.Hkv + h) * bs + off;
          scale_to = (long)new_page * c.Hkv + h;
        }
        if (src < 0 || dst < 0) raise_err(P.err, SD_ERR_KV_RANGE);
      }
      s_src[tid] = src;
      s_dst[tid] = dst;
      s_scale[0][tid] = sk;
      s_scale[1][tid] = sv;
    }
    __syncthreads();
    if (tid < kMoveTokens) {
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {  // (bits of positive numbers are ordered as they are; NaN first)
        const float s = s_scale[kv][tid];
        if (s > 0.f || s != s) atomicMax(&s_max[kv][tid & ~(bs - 1)], __float_as_uint(s) & 0x7fffffffu);
      }
    }
    __syncthreads();
    float new_scale[2] = {0.f, 0.f};
    if (tid < kMoveTokens) {
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const float s = s_scale[kv][tid];
        new_scale[kv] = __uint_as_float(s_max[kv][tid & ~(bs - 1)]);
        const bool none = s_src[tid] < 0 || !(s > 0.f);
        float ratio = none ? 0.f : __fdiv_rn(s, new_scale[kv]);
        if (IN_PLACE && !none && s_src[tid] == s_dst[tid] && ratio == 1.f) ratio = -1.f;
        s_ratio[kv][tid] = ratio;
      }
    }
    __syncthreads();
    // 2. the tokens' bytes: up to 8 parts a thread
    uint4 x[8];
    const int all = 2 * kMoveTokens * parts;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int u = tid + i * kMoveThreads;
      x[i] = make_uint4(0, 0, 0, 0);
      if (u >= all) continue;
      const int kv = u >= kMoveTokens * parts, v = kv ? u - kMoveTokens * parts : u;
      const int t = v / parts, p = v - t * parts;
      if (s_dst[t] >= 0 && (s_ratio[kv][t] > 0.f || s_ratio[kv][t] != s_ratio[kv][t]))
        x[i] = __ldcs(reinterpret_cast<const uint4*>((kv ? P.v : P.k) + s_src[t] + p * 16));
    }
    if (IN_PLACE) cluster_barrier();
    // 3. to their pages
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int u = tid + i * kMoveThreads;
      if (u >= all) continue;
      const int kv = u >= kMoveTokens * parts, v = kv ? u - kMoveTokens * parts : u;
      const int t = v / parts, p = v - t * parts;
      const float ratio = s_ratio[kv][t];
      if (s_dst[t] < 0 || ratio == -1.f) continue;
      if (ratio != 1.f && ratio != 0.f) {
        uint32_t* w = reinterpret_cast<uint32_t*>(&x[i]);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float2 a = e4m3x2_to_f32((uint16_t)w[q]), b = e4m3x2_to_f32((uint16_t)(w[q] >> 16));
          w[q] = f32_to_e4m3x2(a.x * ratio, a.y * ratio) |
                 (uint32_t)f32_to_e4m3x2(b.x * ratio, b.y * ratio) << 16;
        }
      }
      *reinterpret_cast<uint4*>((kv ? P.v : P.k) + s_dst[t] + p * 16) = x[i];
    }
    if (tid < kMoveTokens && weight_to >= 0) {
      P.weights[weight_to] = weight;
      if ((tid & (bs - 1)) == 0) {
        P.k_scale[scale_to] = new_scale[0];
        P.v_scale[scale_to] = new_scale[1];
      }
    }
    if (!IN_PLACE) break;
    __syncthreads();  // (the arrays in shared memory are read)
  }
}

}  // namespace sdk

extern "C" int sd_kv_evict_launch(int B, int Hkv, int D, void* k_cache, void* v_cache,
                                  long st_block, long st_tok, long st_head, float* k_scale,
                                  float* v_scale, int num_blocks, int log2_bs, float* weights,
                                  const int32_t* table, int max_blocks, const int32_t* to_table,
                                  int to_blocks, const int32_t* ctx, int budget, int sink,
                                  int recent, int32_t* kept, int32_t* new_lens, int32_t* err,
                                  cudaStream_t stream) {
  sdk::EvictParams P;
  P.c = sdk::KvCache{(const uint8_t*)k_cache, (const uint8_t*)v_cache, k_scale, v_scale,
                     st_block, st_tok, st_head, num_blocks, log2_bs, Hkv, D};
  P.k = (uint8_t*)k_cache;
  P.v = (uint8_t*)v_cache;
  P.k_scale = k_scale;
  P.v_scale = v_scale;
  P.weights = weights;
  P.B = B;
  P.max_blocks = max_blocks;
  P.to_blocks = to_blocks;
  P.budget = budget;
  P.sink = sink;
  P.recent = recent;
  P.table = table;
  P.to = to_table;
  P.ctx = ctx;
  P.kept = kept;
  P.new_lens = new_lens;
  P.err = err;
  static std::atomic<bool> set[64];  // per device; true only once the attribute is in force
  constexpr int kMostSmem = 200 * 1024;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return SD_E_DEVICE;
  if (!set[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(sdk::evict_choose_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kMostSmem) != cudaSuccess)
      return SD_E_LAUNCH;
    set[dev].store(true, std::memory_order_release);
  }
  const long most = (long)max_blocks << log2_bs;
  P.in_smem = (int)(most < kMostSmem / 4 ? most : kMostSmem / 4);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)Hkv, (unsigned)B, 1);
  cfg.blockDim = dim3(sdk::kSelThreads, 1, 1);
  cfg.dynamicSmemBytes = (size_t)P.in_smem * 4;
  cfg.stream = stream;
  if (cudaLaunchKernelEx(&cfg, sdk::evict_choose_kernel, P) != cudaSuccess) return SD_E_LAUNCH;
  cudaLaunchConfig_t mv = {};
  mv.blockDim = dim3(sdk::kMoveThreads, 1, 1);
  mv.stream = stream;
  if (to_table) {
    const long places = most < budget ? most : budget;
    const unsigned chunks = (unsigned)((places + sdk::kMoveTokens - 1) / sdk::kMoveTokens);
    if (chunks == 0) return SD_OK;
    mv.gridDim = dim3(chunks, (unsigned)Hkv, (unsigned)B);
    return cudaLaunchKernelEx(&mv, sdk::evict_move_kernel<false>, P) == cudaSuccess ? SD_OK
                                                                                   : SD_E_LAUNCH;
  }
  mv.gridDim = dim3(sdk::kMoveCluster, (unsigned)Hkv, (unsigned)B);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = sdk::kMoveCluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  mv.attrs = attr;
  mv.numAttrs = 1;
  return cudaLaunchKernelEx(&mv, sdk::evict_move_kernel<true>, P) == cudaSuccess ? SD_OK
                                                                                : SD_E_LAUNCH;
}
