// sd_evict.cu -- a cache cut to a budget of tokens a request (sd_kv_evict): which tokens stay, by the
// weight that attention has given them, and their move to the front.
//
// Of a request's tokens the first `sink` and the last `recent` stay, and of those between them the
// ones with the largest weights, equal ones in their order, until there are `budget`. Every KV head
// chooses for itself: the heads of a page need not hold the same tokens, only the same number. What
// stays keeps its order; it fills new pages (or the request's own from the first on).

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

constexpr int kSelThreads = 512, kSelWarps = kSelThreads / 32, kSelCluster = 8;

// Tokens that a request's table covers.
__device__ __forceinline__ long evict_covered(const EvictParams& P) {
  return min((long)P.max_blocks << P.c.log2_bs, 2147483647L - 1023);
}
__device__ __forceinline__ int evict_len(const EvictParams& P, int r) {
  const int n = P.ctx[r];
  return n < 0 ? 0 : (int)min((long)n, evict_covered(P));
}

// ---------------------------------------------------------------------------------------------
// Choice: one request and head by a CTA, or by a cluster where there are few of them. The weights become
// orderable keys in shared memory (where they fit, 200 KB; else they are read again), three passes of 11,
// 11 and 10 bits over counts of all CTAs find the last key that stays, and a pass in the tokens' order
// writes down the places. What takes the time is latency: a page and then a weight behind it (eight of
// each on their way a thread), and a dozen barriers. One request of 32000 tokens of 8 heads: 24 us with
// clusters of 8, 69 with a CTA a head; 64 requests of 512 to 8192: 37 us.
// ---------------------------------------------------------------------------------------------
__global__ void __launch_bounds__(kSelThreads) evict_choose_kernel(const EvictParams P) {
  extern __shared__ uint32_t s_key[];
  __shared__ uint32_t s_bin[2][2048];  // counts, by turns of the passes
  __shared__ uint32_t s_warp[kSelWarps], s_warp2[kSelWarps];
  __shared__ uint32_t s_found[2], s_stay[kSelCluster], s_tied[kSelCluster];
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  auto meet = [&]() {
    if (C == 1) __syncthreads();
    else cluster.sync();
  };
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = blockIdx.x / C, r = blockIdx.y;
  const int n = evict_len(P, r), ctx = P.ctx[r];
  const int keep = min(n, P.budget);
  int32_t* kept = P.kept + ((long)r * P.c.Hkv + h) * P.budget;
  if (tid == 0 && h == 0 && rank == 0) {
    P.new_lens[r] = keep;
    if (ctx < 0 || ctx > evict_covered(P)) raise_err(P.err, SD_ERR_KV_RANGE);
  }
  // (budgets and lengths reach 2^31 - 1024, and a cluster's step is up to 4096: 64 bits)
  const long all = C * kSelThreads, me = rank * kSelThreads + tid;
  for (long i = keep + me; i < P.budget; i += all) kept[i] = -1;
  if (n <= P.budget) {
    for (long i = me; i < n; i += all) kept[i] = (int)i;
    return;
  }
  if (C > 1) cluster.sync();  // (every CTA has begun: its shared memory may be written from here on)
  const int32_t* table = P.table + (long)r * P.max_blocks;
  const int bs = 1 << P.c.log2_bs, first = P.sink, m = n - P.sink - P.recent;
  // this CTA's tokens [a0, a1) of those in question
  const int part = (m + C - 1) / C, a0 = min(m, rank * part), a1 = min(m, a0 + part);
  bool bad = false;
  // A token's weight as a key: larger ones first, a NaN before all; one without a page counts as 0.
  auto page_of = [&](int i) { return __ldg(table + ((first + i) >> P.c.log2_bs)); };
  auto key_of = [&](int i, int page) -> uint32_t {
    const bool is = (unsigned)page < (unsigned)P.c.num_blocks;
    bad |= !is;
    float w = 0.f;
    if (is) w = __ldg(P.weights + ((long)page * P.c.Hkv + h) * bs + ((first + i) & (bs - 1)));
    return w != w ? 0xffffffffu : orderable(w);
  };
  const bool held = P.in_smem >= part;
  if (held) {
    for (int i0 = a0 + tid; i0 < a1; i0 += 8 * kSelThreads) {
      int page[8];
      uint32_t k[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) page[j] = i0 + j * kSelThreads < a1 ? page_of(i0 + j * kSelThreads) : 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) k[j] = i0 + j * kSelThreads < a1 ? key_of(i0 + j * kSelThreads, page[j]) : 0;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (i0 + j * kSelThreads < a1) s_key[i0 + j * kSelThreads - a0] = k[j];
    }
  }
  auto key = [&](int i) { return held ? s_key[i - a0] : key_of(i, page_of(i)); };

  uint32_t need = (uint32_t)(P.budget - P.sink - P.recent);  // < m
  uint32_t prefix = 0;
  const bool any = need > 0;
  for (int level = 0; any && level < 3; ++level) {
    const int shift = level == 0 ? 21 : level == 1 ? 10 : 0, bits = level == 2 ? 10 : 11;
    const uint32_t high = level == 0 ? 0u : 0xffffffffu << (shift + bits);
    uint32_t* bin = s_bin[level & 1];
    for (int i = tid; i < 2048; i += kSelThreads) bin[i] = 0;
    __syncthreads();
    for (int i = a0 + tid; i < a1; i += kSelThreads) {
      const uint32_t k = key(i);
      if ((k & high) == prefix) atomicAdd(&bin[2047 - ((k >> shift) & ((1u << bits) - 1))], 1u);
    }
    meet();
    // the bin in which number `need` from the largest lies: 4 bins a thread, of all CTAs
    uint32_t c[4], sum = 0;
    {
      uint4 v = reinterpret_cast<const uint4*>(bin)[tid];
      if (C > 1) {
        v = make_uint4(0, 0, 0, 0);
        for (int k = 0; k < C; ++k) {
          const uint4 x = reinterpret_cast<const uint4*>(cluster.map_shared_rank(bin, k))[tid];
          v.x += x.x;
          v.y += x.y;
          v.z += x.z;
          v.w += x.w;
        }
      }
      c[0] = v.x;
      c[1] = v.y;
      c[2] = v.z;
      c[3] = v.w;
      sum = v.x + v.y + v.z + v.w;
    }
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

  // the places, in order: a warp goes over a stretch of its own, of this CTA's part with the tokens
  // before it (the first CTA) and behind it (the last one)
  const int b0 = rank == 0 ? 0 : first + a0, b1 = rank == C - 1 ? n : first + a1;
  const int seg = (b1 - b0 + kSelWarps * 32 - 1) / (kSelWarps * 32) * 32;
  const int a = min(b1, b0 + warp * seg), b = min(b1, a + seg);
  // 0: goes, 1: stays, 2: stays if it is among the first `ties` of its key
  auto kind = [&](int t) {
    if (t < P.sink || t >= n - P.recent) return 1;
    if (!any) return 0;
    const uint32_t k = key(t - first);
    return k > prefix ? 1 : k == prefix ? 2 : 0;
  };
  uint32_t stay = 0, tied = 0;
#pragma unroll 4
  for (int i = a; i < b; i += 32) {
    const int x = i + lane < b ? kind(i + lane) : 0;
    stay += x == 1;
    tied += x == 2;
  }
  stay = __reduce_add_sync(0xffffffffu, stay);
  tied = __reduce_add_sync(0xffffffffu, tied);
  if (lane == 0) {
    s_warp[warp] = stay;
    s_warp2[warp] = tied;
  }
  __syncthreads();
  if (C > 1) {
    if (tid < C) {
      uint32_t x = 0, y = 0;
      for (int w = 0; w < kSelWarps; ++w) {
        x += s_warp[w];
        y += s_warp2[w];
      }
      cluster.map_shared_rank(s_stay, tid)[rank] = x;
      cluster.map_shared_rank(s_tied, tid)[rank] = y;
    }
    cluster.sync();
  }
  stay = tied = 0;
  for (int k = 0; k < rank; ++k) {
    stay += s_stay[k];
    tied += s_tied[k];
  }
  for (int w = 0; w < warp; ++w) {
    stay += s_warp[w];
    tied += s_warp2[w];
  }
  const uint32_t below = (1u << lane) - 1;
#pragma unroll 2
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
// Move: a CTA takes 128 places (whole pages; 256 of heads of up to 64) of one head, first K and then V,
// into registers and then to their new pages. A new page's scale is the largest of its tokens' (their sources' pages'), so that
// values only ever lose what becomes subnormal, and a page of tokens that do not move stays as it is.
// Within the request's own pages a token only moves towards the front: a cluster goes over the
// places in rounds, and nothing is written before all of the round's tokens are read. Bound by memory
// behind a chain of three loads (place, page, scale): 64 requests of up to 2048 tokens of 8 heads of 64
// take 60 us, 66% of the copy rate (K and V together in registers, four CTAs an SM instead of five: 79);
// one request of 16000 of 128 16 us. Within their own pages the whole calls take 101 us (98 into fresh
// ones) and 105 (31 to 39): a cluster a head goes over the one request's places in 16 rounds.
// ---------------------------------------------------------------------------------------------
constexpr int kMoveThreads = 256, kMoveCluster = 8;

template <bool IN_PLACE, int kMoveTokens>
__global__ void __launch_bounds__(kMoveThreads, 5) evict_move_kernel(const EvictParams P) {
  __shared__ long s_src[kMoveTokens], s_dst[kMoveTokens];  // elements; -1: no page, -2: no token
  __shared__ float s_scale[2][kMoveTokens];
  __shared__ unsigned s_max[2][kMoveTokens];  // of each page, in its first token's place
  __shared__ float s_ratio[2][kMoveTokens];   // -1: stays as it is
  asm volatile("griddepcontrol.wait;" ::: "memory");  // (the places)
  const KvCache& c = P.c;
  const int tid = threadIdx.x, h = blockIdx.y, r = blockIdx.z;
  const int n = min(evict_len(P, r), P.budget), bs = 1 << c.log2_bs;
  const int32_t* kept = P.kept + ((long)r * c.Hkv + h) * P.budget;
  const int32_t* table = P.table + (long)r * P.max_blocks;
  const int32_t* to = IN_PLACE ? table : P.to + (long)r * P.to_blocks;
  const int to_blocks = IN_PLACE ? P.max_blocks : P.to_blocks;
  const int parts = c.D / 16;  // 16-byte parts of a token's head
  if (!IN_PLACE && (long)blockIdx.x * kMoveTokens >= n) return;
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
    // 2. the tokens' bytes, 4 parts a thread, and on to their pages
    const int all = kMoveTokens * parts;
#pragma unroll 1
    for (int kv = 0; kv < 2; ++kv) {
      uint8_t* cache = kv ? P.v : P.k;
      uint4 x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int u = tid + i * kMoveThreads, t = u / parts;
        x[i] = make_uint4(0, 0, 0, 0);
        if (u < all && s_dst[t] >= 0 && (s_ratio[kv][t] > 0.f || s_ratio[kv][t] != s_ratio[kv][t]))
          x[i] = __ldcs(reinterpret_cast<const uint4*>(cache + s_src[t] + (u - t * parts) * 16));
      }
      if (IN_PLACE) cluster_barrier();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int u = tid + i * kMoveThreads, t = u / parts;
        if (u >= all) continue;
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
        *reinterpret_cast<uint4*>(cache + s_dst[t] + (u - t * parts) * 16) = x[i];
      }
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

template <int TOKENS>
static int launch_move(const EvictParams& P, long most, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.blockDim = dim3(kMoveThreads, 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (P.to) {
    const long places = most < P.budget ? most : P.budget;
    const unsigned chunks = (unsigned)((places + TOKENS - 1) / TOKENS);
    if (chunks == 0) return SD_OK;
    cfg.gridDim = dim3(chunks, (unsigned)P.c.Hkv, (unsigned)P.B);
    return cudaLaunchKernelEx(&cfg, evict_move_kernel<false, TOKENS>, P) == cudaSuccess ? SD_OK
                                                                                       : SD_E_LAUNCH;
  }
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kMoveCluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.numAttrs = 2;
  cfg.gridDim = dim3(kMoveCluster, (unsigned)P.c.Hkv, (unsigned)P.B);
  return cudaLaunchKernelEx(&cfg, evict_move_kernel<true, TOKENS>, P) == cudaSuccess ? SD_OK
                                                                                     : SD_E_LAUNCH;
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
  static std::atomic<bool> set[sdk::kMostDevices];  // per device; true only once the attribute is in force
  constexpr int kMostSmem = 200 * 1024;
  int dev = 0;
  const int sms = sdk::device_sms(dev);
  if (sms == 0) return SD_E_DEVICE;
  if (!set[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(sdk::evict_choose_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kMostSmem) != cudaSuccess)
      return SD_E_LAUNCH;
    set[dev].store(true, std::memory_order_release);
  }
  const long most = (long)max_blocks << log2_bs;
  // CTAs of a request and head: more while the SMs have room for them and each has 1000 tokens. (512
  // requests and heads with 1, 2, 4: the call 102, 120, 168 us; 8 with 1 and 8: 85 and 39.)
  int C = 1;
  while (C < sdk::kSelCluster && (long)B * Hkv * C * 2 <= 2 * sms && most > 2048L * C) C *= 2;
  const long part = (most + C - 1) / C;
  P.in_smem = (int)(part < kMostSmem / 4 ? part : kMostSmem / 4);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)C;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)(Hkv * C), (unsigned)B, 1);
  cfg.blockDim = dim3(sdk::kSelThreads, 1, 1);
  cfg.dynamicSmemBytes = (size_t)P.in_smem * 4;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, sdk::evict_choose_kernel, P) != cudaSuccess) return SD_E_LAUNCH;
  return D <= 64 ? sdk::launch_move<256>(P, most, stream) : sdk::launch_move<128>(P, most, stream);
}
