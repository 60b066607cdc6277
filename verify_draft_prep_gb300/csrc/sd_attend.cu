// sd_attend.cu -- attention over the paged 8-bit cache (sd_kv_attend).
//
// Query token i of request r stands at position ctx_lens[r] - n_q + i and sees every token up to
// its own position (causal) or all ctx_lens[r] tokens. With S = sm_scale q k and the running
// maximum M and sum L of its exponentials, O = sum e^(S - M) v / L and lse = M + ln L.

#include "sd_kv.cuh"

namespace sdk {

struct AttendParams {
  KvCache c;
  int B, n, Hq, max_blocks, causal;
  const uint16_t* q;
  long ld_q, hs_q;
  const int32_t* table;
  const int32_t* ctx;
  const int32_t* cu;
  float scale;
  uint16_t* out;
  long ld_out, hs_out;
  float* lse;
  int32_t* err;
};

// One warp for a query token and head: 32 tokens of the cache at a time, one a lane for the
// scores, then the lanes share the head's dimensions for the weighted sum.
__global__ void __launch_bounds__(256) attend_simple_kernel(const AttendParams P) {
  const KvCache& c = P.c;
  const int lane = threadIdx.x & 31;
  const long w = (long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int i = (int)(w / P.Hq), hq = (int)(w % P.Hq), h = hq / (P.Hq / c.Hkv);
  if (i >= P.n || i < P.cu[0] || i >= P.cu[P.B]) return;
  int lo = 0, hi = P.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (P.cu[mid] <= i) lo = mid;
    else hi = mid;
  }
  const long cover = (long)P.max_blocks << c.log2_bs;
  long len = P.ctx[lo];
  if (len < 0 || len > cover) {
    raise_err(P.err, SD_ERR_KV_RANGE);
    len = len < 0 ? 0 : cover;
  }
  const int begin = max(P.cu[lo], 0), end = min(P.cu[lo + 1], P.n);
  if (begin != P.cu[lo] || end != P.cu[lo + 1]) raise_err(P.err, SD_ERR_KV_RANGE);
  const long pos = (long)P.ctx[lo] - (end - begin) + (i - begin);
  const long seen = P.causal ? min(len, pos + 1) : len;
  __shared__ float s_q[8][128];
  float* q = s_q[threadIdx.x >> 5];
  for (int d = lane; d < c.D; d += 32)
    q[d] = __uint_as_float((uint32_t)P.q[i * P.ld_q + hq * P.hs_q + d] << 16) * P.scale;
  __syncwarp();
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  for (long t0 = 0; t0 < seen; t0 += 32) {
    const long t = t0 + lane;
    float s = -INFINITY, vs = 0.f;
    long base = 0;
    if (t < seen) {
      const int page = P.table[(long)lo * P.max_blocks + (t >> c.log2_bs)];
      if (page >= 0 && page < c.num_blocks) {
        base = page * c.st_block + (t & ((1 << c.log2_bs) - 1)) * c.st_tok + h * c.st_head;
        s = 0.f;
        for (int d = 0; d < c.D; d += 2) {
          const float2 k = e4m3x2_to_f32(*reinterpret_cast<const uint16_t*>(c.k + base + d));
          s += q[d] * k.x + q[d + 1] * k.y;
        }
        s *= c.k_scale[(long)page * c.Hkv + h];
        vs = c.v_scale[(long)page * c.Hkv + h];
      } else {
        raise_err(P.err, SD_ERR_KV_RANGE);
      }
    }
    float mx = s;
    for (int x = 16; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
    const float mn = fmaxf(m, mx);
    const float e = s == -INFINITY ? 0.f : expf(s - mn);
    const float f = m == -INFINITY ? 0.f : expf(m - mn);
    float sum = e;
    for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
    l = l * f + sum;
    m = mn;
    for (int k = 0; k < 4; ++k) o[k] *= f;
    for (int j = 0; j < 32; ++j) {
      const float pj = __shfl_sync(0xffffffffu, e, j) * __shfl_sync(0xffffffffu, vs, j);
      const float sj = __shfl_sync(0xffffffffu, s, j);
      const long bj = __shfl_sync(0xffffffffu, base, j);
      if (sj == -INFINITY) continue;
      for (int k = 0; k < 4; ++k) {
        const int d = lane + 32 * k;
        if (d < c.D) o[k] += pj * e4m3x2_to_f32(c.v[bj + d]).x;
      }
    }
  }
  for (int k = 0; k < 4; ++k) {
    const int d = lane + 32 * k;
    if (d < c.D) {
      const __nv_bfloat16 r = __float2bfloat16_rn(l == 0.f ? 0.f : o[k] / l);
      P.out[i * P.ld_out + hq * P.hs_out + d] = *reinterpret_cast<const uint16_t*>(&r);
    }
  }
  if (P.lse && lane == 0) P.lse[(long)i * P.Hq + hq] = l == 0.f ? -INFINITY : m + logf(l);
}

}  // namespace sdk

extern "C" size_t sd_kv_attend_workspace_launch(int D) {
  (void)D;
  return 0;
}

extern "C" int sd_kv_attend_launch(int B, int n, int max_q, int Hq, int Hkv, int D, const void* q,
                                   long ld_q, long hs_q, const void* k_cache, const void* v_cache,
                                   long st_block, long st_tok, long st_head, const float* k_scale,
                                   const float* v_scale, int num_blocks, int log2_bs,
                                   const int32_t* table, int max_blocks, const int32_t* ctx,
                                   const int32_t* cu, float sm_scale, int causal, void* out,
                                   long ld_out, long hs_out, float* lse, void* workspace,
                                   int32_t* err, cudaStream_t stream) {
  (void)max_q;
  (void)workspace;
  sdk::AttendParams P;
  P.c = sdk::KvCache{(const uint8_t*)k_cache, (const uint8_t*)v_cache, k_scale, v_scale,
                     st_block, st_tok, st_head, num_blocks, log2_bs, Hkv, D};
  P.B = B;
  P.n = n;
  P.Hq = Hq;
  P.max_blocks = max_blocks;
  P.causal = causal;
  P.q = (const uint16_t*)q;
  P.ld_q = ld_q;
  P.hs_q = hs_q;
  P.table = table;
  P.ctx = ctx;
  P.cu = cu;
  P.scale = sm_scale;
  P.out = (uint16_t*)out;
  P.ld_out = ld_out;
  P.hs_out = hs_out;
  P.lse = lse;
  P.err = err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(((long)n * Hq + 7) / 8), 1, 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.stream = stream;
  return cudaLaunchKernelEx(&cfg, sdk::attend_simple_kernel, P) == cudaSuccess ? SD_OK
                                                                               : SD_E_LAUNCH;
}
