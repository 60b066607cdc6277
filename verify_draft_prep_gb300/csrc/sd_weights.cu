// sd_weights.cu -- the attention weight that each cached token gets from a call's queries
// (sd_kv_weights).
//
// w[t] = sum over the query tokens i that count and the heads g of the group, of those that see t,
// e^(sm_scale q_ig . k_t - lse_ig), added to `decay` times what t had before (nothing for the call's
// own tokens). A CTA has 128 tokens of one KV head, a token a thread, and goes over all rows (a row is
// a query token and a head), so that every sum has one owner and a fixed order.

#include "sd_kv.cuh"

namespace sdk {

struct WeightsParams {
  KvCache c;
  int B, n, Hq, G, max_blocks, causal;
  const uint16_t* q;
  long ld_q, hs_q;
  const float* lse;
  const int32_t* table;
  const int32_t* ctx;
  const int32_t* cu;
  const int32_t* live;
  float scale;  // sm_scale * log2(e)
  float decay;
  const float* before;
  float* weights;
  int32_t* err;
};

constexpr int kWTile = 128, kWRows = 32;

template <int DP>
__global__ void __launch_bounds__(kWTile) weights_simple_kernel(const WeightsParams P) {
  __shared__ float s_q[kWRows][DP];
  __shared__ float s_lse[kWRows];
  const KvCache& c = P.c;
  const int tid = threadIdx.x, h = blockIdx.y, r = blockIdx.z, bs = 1 << c.log2_bs;
  const int a = P.cu[r], b = P.cu[r + 1];
  const int lo = min(max(a, 0), P.n), hi = min(max(b, lo), P.n), n_q = hi - lo;
  const int ctx = P.ctx[r];
  const long covered = min((long)P.max_blocks << c.log2_bs, 2147483648L - 256);
  const int len = ctx < 0 ? 0 : (int)min((long)ctx, covered);
  const long off = (long)ctx - n_q;
  int live = P.live ? P.live[r] : n_q;
  if (tid == 0 && blockIdx.x == 0 && h == 0 &&
      (a < 0 || b < a || b > P.n || ctx < 0 || ctx > covered || live < 0 || live > n_q))
    raise_err(P.err, SD_ERR_KV_RANGE);
  live = min(max(live, 0), n_q);
  if ((long)blockIdx.x * kWTile >= len) return;
  const int t = blockIdx.x * kWTile + tid;
  int page = -1;
  if (t < len) {
    page = P.table[(long)r * P.max_blocks + (t >> c.log2_bs)];
    if ((unsigned)page >= (unsigned)c.num_blocks) {
      page = -1;
      raise_err(P.err, SD_ERR_KV_RANGE);
    }
  }
  float k[DP];
  float ks = 0.f;
  if (page >= 0) ks = c.k_scale[(long)page * c.Hkv + h];
#pragma unroll
  for (int d = 0; d < DP; d += 16) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (page >= 0 && d < c.D && ks != 0.f)
      v = __ldg(reinterpret_cast<const uint4*>(c.k + page * c.st_block + (t & (bs - 1)) * c.st_tok +
                                               h * c.st_head + d));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = e4m3x2_to_f32((uint16_t)w[i]), y = e4m3x2_to_f32((uint16_t)(w[i] >> 16));
      k[d + 4 * i] = x.x;
      k[d + 4 * i + 1] = x.y;
      k[d + 4 * i + 2] = y.x;
      k[d + 4 * i + 3] = y.y;
    }
  }
  const float f = ks * P.scale;
  float sum = 0.f, rest = 0.f;  // (compensated)
  const int rows = live * P.G;
  for (int r0 = 0; r0 < rows; r0 += kWRows) {
    __syncthreads();
    for (int i = tid; i < kWRows * DP; i += kWTile) {
      const int row = r0 + i / DP, d = i % DP;
      float x = 0.f;
      if (row < rows && d < c.D)
        x = bf16_bits_to_float(P.q[(long)(lo + row / P.G) * P.ld_q +
                                   (long)(h * P.G + row % P.G) * P.hs_q + d]);
      s_q[i / DP][d] = x;
    }
    if (tid < kWRows && r0 + tid < rows)
      s_lse[tid] = P.lse[(long)(lo + (r0 + tid) / P.G) * P.Hq + h * P.G + (r0 + tid) % P.G];
    __syncthreads();
    const int m = min(kWRows, rows - r0);
    float part = 0.f;
    for (int i = 0; i < m; ++i) {
      if (P.causal && t > off + (r0 + i) / P.G) continue;
      float s = 0.f;
#pragma unroll
      for (int d = 0; d < DP; d += 4) {
        const float4 v = *reinterpret_cast<const float4*>(&s_q[i][d]);
        s = fmaf(v.x, k[d], s);
        s = fmaf(v.y, k[d + 1], s);
        s = fmaf(v.z, k[d + 2], s);
        s = fmaf(v.w, k[d + 3], s);
      }
      part += exp2f(s * f - s_lse[i] * 1.4426950408889634f);
    }
    const float y = part - rest, z = sum + y;
    rest = (z - sum) - y;
    sum = z;
  }
  if (page >= 0) {
    const long at = ((long)page * c.Hkv + h) * bs + (t & (bs - 1));
    P.weights[at] = P.before && t < off ? fmaf(P.decay, P.before[at], sum) : sum;
  }
}

}  // namespace sdk

extern "C" int sd_kv_weights_launch(int B, int n, int max_q, int Hq, int Hkv, int D, const void* q,
                                    long ld_q, long hs_q, const float* lse, const void* k_cache,
                                    long st_block, long st_tok, long st_head,
                                    const float* k_scale, int num_blocks, int log2_bs,
                                    const int32_t* table, int max_blocks, const int32_t* ctx,
                                    const int32_t* cu, const int32_t* live, float sm_scale,
                                    int causal, float decay, const float* before, float* weights,
                                    int32_t* err, cudaStream_t stream) {
  sdk::WeightsParams P;
  P.c = sdk::KvCache{(const uint8_t*)k_cache, nullptr, k_scale, nullptr,
                     st_block, st_tok, st_head, num_blocks, log2_bs, Hkv, D};
  P.B = B;
  P.n = n;
  P.Hq = Hq;
  P.G = Hq / Hkv;
  P.max_blocks = max_blocks;
  P.causal = causal;
  P.q = (const uint16_t*)q;
  P.ld_q = ld_q;
  P.hs_q = hs_q;
  P.lse = lse;
  P.table = table;
  P.ctx = ctx;
  P.cu = cu;
  P.live = live;
  P.scale = sm_scale * 1.4426950408889634f;
  P.decay = decay;
  P.before = before;
  P.weights = weights;
  P.err = err;
  (void)max_q;
  const long tiles = (((long)max_blocks << log2_bs) + sdk::kWTile - 1) / sdk::kWTile;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles > 0 ? tiles : 1), (unsigned)Hkv, (unsigned)B);
  cfg.blockDim = dim3(sdk::kWTile, 1, 1);
  cfg.stream = stream;
  return (D <= 64 ? cudaLaunchKernelEx(&cfg, sdk::weights_simple_kernel<64>, P)
                  : cudaLaunchKernelEx(&cfg, sdk::weights_simple_kernel<128>, P)) == cudaSuccess
             ? SD_OK
             : SD_E_LAUNCH;
}
