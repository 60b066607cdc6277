// sd_kv.cu -- the paged 8-bit cache: quantised as it is written (sd_kv_write), read back
// (sd_kv_read).
//
// A page (block_size tokens) and head has one scale s, a power of two, and holds e4m3(x / s). e4m3
// is a floating type, so a power of two as scale loses no relative precision against amax / 448,
// every product with it is exact, and a page rounded again to a larger scale (because a later
// token needs one) changes only where values become subnormal.

#include "sd_kv.cuh"

namespace sdk {

// ---------------------------------------------------------------------------------------------
// Write. A run is the tokens of one page in one call (they stand next to one another in the slot
// mapping, up to 31 entries that are not written between them). A page of up to 16 tokens of one
// head of K or V is one warp's work, so that the page stays in registers between the largest
// magnitude and the quantisation: every value is read once. Larger pages take a team of warps, 16
// tokens each, that meet over the magnitude. Per element 2 bytes are read and 1 is written; the
// kernel is bound by memory for prompts (2 x 8192 tokens of 8 heads of 128: 18.7 us in a graph, 79%
// of the copy rate; 1024 CTAs on 608 places, so that the second wave is not full) and by the chain
// slot -> token -> scale -> store for the few tokens of a step (64 requests of 6 tokens of 8 heads
// of 64: 6.3 us in a graph).
// ---------------------------------------------------------------------------------------------
struct KvWriteParams {
  const uint16_t* x[2];  // K, V rows
  long ld[2], hs[2];
  uint8_t* cache[2];
  float* scale[2];
  long st_block, st_tok, st_head;
  int n, Hkv, D, num_blocks, log2_bs, chunk;
  const int32_t* slots;
  int32_t* err;
};

constexpr int kWriteThreads = 256;

// The smallest power of two s >= 2^-100 with a <= 448 s. a = m 2^e with m in [0.5, 1), and
// 448 = 0.875 * 2^9.
__device__ __forceinline__ float pow2_scale(float a) {
  const uint32_t b = __float_as_uint(a);
  const int e = (int)(b >> 23) - 126;
  const int k = e - 9 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return k <= -100 ? kMinScale : __uint_as_float((uint32_t)(k + 127) << 23);
}

// The largest finite of 8 bf16 magnitudes, as a 16-bit pattern (infinities and NaN count as 0).
__device__ __forceinline__ uint32_t finite_max(const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = w[i] & 0x7fffu, hi = (w[i] >> 16) & 0x7fffu;
    m = max(m, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
  }
  return m;
}

// 8 bf16 times r (exact: r a power of two), or over s where r is 0, as e4m3 to nearest even.
__device__ __forceinline__ uint2 quant8(const uint4& v, float r, float s) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o[i] = r > 0.f ? f32_to_e4m3x2(bf16_lo(w[i]) * r, bf16_hi(w[i]) * r)
                   : f32_to_e4m3x2(__fdiv_rn(bf16_lo(w[i]), s), __fdiv_rn(bf16_hi(w[i]), s));
  return make_uint2(o[0] | o[1] << 16, o[2] | o[3] << 16);
}

__global__ void __launch_bounds__(kWriteThreads, 4) kv_write_kernel(const KvWriteParams P) {
  extern __shared__ int32_t s_map[];  // [runs of this CTA][block_size]: the token of each slot
  __shared__ int32_t s_lead[32];
  __shared__ int s_runs;
  __shared__ uint32_t s_mag[kWriteThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int bs = 1 << P.log2_bs;
  const int i0 = blockIdx.x * P.chunk;
  const long limit = (long)P.num_blocks << P.log2_bs;
  auto written = [&](int s) { return s < limit ? s : -1; };  // a slot, or -1

  // 1. The runs that begin in this CTA's tokens.
  if (warp == 0) {
    bool lead = false, bad = false;
    if (lane < P.chunk && i0 + lane < P.n) {
      const int s = P.slots[i0 + lane];
      int prev = i0 + lane > 0 ? written(P.slots[i0 + lane - 1]) : -1;
      bad = s >= limit;
      if (s >= 0 && !bad) {
        // the last slot before this one, over up to 31 that are not written
        for (int j = i0 + lane - 2; j >= 0 && j >= i0 + lane - 32 && prev < 0; --j)
          prev = written(P.slots[j]);
        lead = prev < 0 || (prev >> P.log2_bs) != (s >> P.log2_bs);
      }
    }
    const uint32_t m = __ballot_sync(0xffffffffu, lead);
    if (lead) s_lead[__popc(m & ((1u << lane) - 1))] = i0 + lane;
    if (lane == 0) s_runs = __popc(m);
    if (bad && blockIdx.y == 0) raise_err(P.err, SD_ERR_KV_SLOT);
  }
  __syncthreads();
  const int runs = s_runs;
  if (runs == 0) return;

  // 2. Slot -> token of each run (of tokens that share a slot, the last one).
  for (int i = tid; i < runs << P.log2_bs; i += kWriteThreads) s_map[i] = -1;
  __syncthreads();
  for (int r = warp; r < runs; r += kWriteThreads / 32) {
    const int first = s_lead[r];
    const int page = P.slots[first] >> P.log2_bs;
    for (int i = first; i < P.n;) {
      const int s = i + lane < P.n ? written(P.slots[i + lane]) : -1;
      const bool here = s >= 0 && (s >> P.log2_bs) == page;
      const uint32_t other = __ballot_sync(0xffffffffu, s >= 0 && !here);
      const int len = other ? __ffs(other) - 1 : 32;
      const uint32_t in = __ballot_sync(0xffffffffu, here && lane < len);
      if (here && lane < len) atomicMax(&s_map[(r << P.log2_bs) + (s & (bs - 1))], i + lane);
      if (other || !in) break;
      i += 32 - __clz(in);  // on behind the last token of the page
    }
  }
  __syncthreads();

  // 3. One team of warps for each (run, K or V, head).
  const int team_warps = bs > 16 ? bs / 16 : 1;
  const int teams = (kWriteThreads / 32) / team_warps;
  const int team = warp / team_warps, sub = warp % team_warps;
  const int row_lanes = P.D / 8;                // lanes that hold one token's head, 8 values each
  const int rows = 32 / row_lanes;              // tokens of one of its 8 register sets, 2 or more
  const int my_row = lane / row_lanes, col = lane % row_lanes;
  const int slots = bs < 16 ? bs : 16;          // slots of the page that this warp holds
  const int pairs = 2 * P.Hkv;
  const int work = runs * pairs;
  for (int w0 = blockIdx.y * teams; w0 < work; w0 += gridDim.y * teams) {
    const int w = w0 + team;
    const bool active = w < work;
    const int run = active ? w / pairs : 0, pair = active ? w % pairs : 0;
    const int kv = pair / P.Hkv, h = pair % P.Hkv;
    const int32_t* map = s_map + (run << P.log2_bs);
    const int page = P.slots[s_lead[run]] >> P.log2_bs;
    float* sp = P.scale[kv] + (long)page * P.Hkv + h;
    uint8_t* base = P.cache[kv] + page * P.st_block + h * P.st_head + col * 8;

    uint4 x[8];
    uint32_t mag = 0, have = 0;  // have: the sets of which this lane holds a token of the call
#pragma unroll
    for (int it = 0; it < 8; ++it) {
      const int j = it * rows + my_row;
      x[it] = make_uint4(0, 0, 0, 0);
      if (active && my_row < rows && j < slots) {
        const int t = map[sub * 16 + j];
        if (t >= 0) have |= 1u << it;
        if (t >= 0)
          x[it] = __ldcs(reinterpret_cast<const uint4*>(P.x[kv] + t * P.ld[kv] + h * P.hs[kv] +
                                                        col * 8));
      }
    }
    float s_old = active ? *sp : 0.f;
#pragma unroll
    for (int it = 0; it < 8; ++it) {
      mag = __vmaxu2(mag, __vmaxu2(__vmaxu2(x[it].x & 0x7fff7fffu, x[it].y & 0x7fff7fffu),
                                   __vmaxu2(x[it].z & 0x7fff7fffu, x[it].w & 0x7fff7fffu)));
    }
    mag = __reduce_max_sync(0xffffffffu, max(mag & 0xffffu, mag >> 16));
    if (mag >= 0x7f80u) {  // an infinity or a NaN: rare, and it does not enter the scale
      mag = 0;
#pragma unroll
      for (int it = 0; it < 8; ++it) mag = max(mag, finite_max(x[it]));
      mag = __reduce_max_sync(0xffffffffu, mag);
    }
    if (team_warps > 1) {
      __syncthreads();  // the last round's magnitudes are read, and every scale of this round
      if (lane == 0) s_mag[warp] = mag;
      __syncthreads();
      for (int i = 0; i < team_warps; ++i) mag = max(mag, s_mag[team * team_warps + i]);
    }
    if (!active) continue;
    const bool fresh = map[0] >= 0;
    if (!(s_old > 0.f)) s_old = 0.f;
    const float held = fresh ? 0.f : s_old;
    const float s = fmaxf(held, pow2_scale(__uint_as_float(mag << 16)));
    if (sub == 0 && lane == 0) *sp = s;
    const float r = __fdiv_rn(1.f, s);
    const float inv = (__float_as_uint(s) & 0x7fffffu) == 0 && r >= 1.17549435e-38f ? r : 0.f;
    const bool again = !fresh && s != s_old;
    const float ratio = __fdiv_rn(s_old, s);
    if (inv > 0.f) {
#pragma unroll
      for (int it = 0; it < 8; ++it)
        if ((have >> it) & 1)
          *reinterpret_cast<uint2*>(base + (sub * 16 + it * rows + my_row) * P.st_tok) =
              quant8(x[it], inv, s);
    } else {
#pragma unroll
      for (int it = 0; it < 8; ++it)
        if ((have >> it) & 1)
          *reinterpret_cast<uint2*>(base + (sub * 16 + it * rows + my_row) * P.st_tok) =
              quant8(x[it], 0.f, s);
    }
    if (again) {  // what the page held in its other slots, at its new scale
#pragma unroll 1
      for (int it = 0; it < 8; ++it) {
        if (my_row >= rows || it * rows + my_row >= slots || (have >> it) & 1) continue;
        uint2* dst =
            reinterpret_cast<uint2*>(base + (sub * 16 + it * rows + my_row) * P.st_tok);
        // (a page of scale 0 holds zeros, whatever its bytes)
        const uint2 q = s_old > 0.f ? *dst : make_uint2(0, 0);
        uint32_t o[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t qi = i ? q.y : q.x;
          const float2 a = e4m3x2_to_f32((uint16_t)qi), b = e4m3x2_to_f32((uint16_t)(qi >> 16));
          o[i] = f32_to_e4m3x2(a.x * ratio, a.y * ratio) |
                 (uint32_t)f32_to_e4m3x2(b.x * ratio, b.y * ratio) << 16;
        }
        *dst = make_uint2(o[0], o[1]);
      }
    }
  }
}

// ---------------------------------------------------------------------------------------------
// Read back. Output row i is token i - cu[r] + first[r] of request r. A CTA takes 16 rows: their
// pages are looked up once into shared memory (a binary search over the prefix), then every thread
// moves 16 values at a time (16 bytes in, 32 out), four of them on their way. Bound by memory, 1
// byte read and 2 written for each value: 316000 tokens of 8 heads of 64 take 147 us, 97% of the
// copy rate; one request of 32000 tokens of 8 heads of 128 36 us, 79%: 2000 CTAs on 912 places, the
// third wave a fifth full.
// ---------------------------------------------------------------------------------------------
struct KvReadParams {
  KvCache c;
  int B, n, max_blocks;
  const int32_t* table;
  const int32_t* cu;
  const int32_t* first;
  uint16_t* out[2];
  long ld, hs;
  int32_t* err;
};

constexpr int kReadThreads = 256, kReadRows = 16;

__device__ __forceinline__ uint32_t scaled_bf16x2(uint16_t q, float s) {
  const float2 f = e4m3x2_to_f32(q);
  const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * s, f.y * s);
  return *reinterpret_cast<const uint32_t*>(&b);
}

__global__ void __launch_bounds__(kReadThreads) kv_read_kernel(const KvReadParams P) {
  __shared__ int s_page[kReadRows], s_off[kReadRows];
  const KvCache& c = P.c;
  const int tid = threadIdx.x;
  const int i0 = blockIdx.x * kReadRows;
  if (tid < kReadRows) {
    const int i = i0 + tid;
    int page = -2, off = 0;  // -2: not a row of any request
    if (i < P.n && i >= P.cu[0] && i < P.cu[P.B]) {
      int lo = 0, hi = P.B;  // the last r with cu[r] <= i
      while (hi - lo > 1) {
        const int mid = lo + ((hi - lo) >> 1);
        if (P.cu[mid] <= i) lo = mid;
        else hi = mid;
      }
      const long pos = (long)i - P.cu[lo] + (P.first ? P.first[lo] : 0);
      const long b = pos >> c.log2_bs;
      page = -1;
      if (pos >= 0 && b < P.max_blocks) {
        page = P.table[(long)lo * P.max_blocks + b];
        if (page >= c.num_blocks) page = -1;
      }
      if (page < 0) {
        page = -1;
        raise_err(P.err, SD_ERR_KV_RANGE);
      }
      off = (int)(pos & ((1 << c.log2_bs) - 1));
    }
    s_page[tid] = page;
    s_off[tid] = off;
  }
  __syncthreads();
  const int parts = c.D / 16, per_row = c.Hkv * parts;
#pragma unroll 4
  for (int u = tid; u < kReadRows * per_row; u += kReadThreads) {
    const int row = u / per_row, e = u % per_row, h = e / parts, d = (e % parts) * 16;
    const int page = s_page[row];
    if (page == -2) continue;
    const long dst = (long)(i0 + row) * P.ld + h * P.hs + d;
    const long src = page * c.st_block + s_off[row] * c.st_tok + h * c.st_head + d;
    uint4 q[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    float s[2] = {0.f, 0.f};
    if (page >= 0) {
      q[0] = __ldcs(reinterpret_cast<const uint4*>(c.k + src));
      q[1] = __ldcs(reinterpret_cast<const uint4*>(c.v + src));
      s[0] = c.k_scale[(long)page * c.Hkv + h];
      s[1] = c.v_scale[(long)page * c.Hkv + h];
    }
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      const uint32_t keep = s[kv] == 0.f ? 0u : ~0u;  // a scale of 0: zeros, whatever the bytes
      const uint32_t w[4] = {q[kv].x & keep, q[kv].y & keep, q[kv].z & keep, q[kv].w & keep};
      uint32_t o[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        o[2 * k] = scaled_bf16x2((uint16_t)w[k], s[kv]);
        o[2 * k + 1] = scaled_bf16x2((uint16_t)(w[k] >> 16), s[kv]);
      }
      uint4* p = reinterpret_cast<uint4*>(P.out[kv] + dst);
      __stcs(p, make_uint4(o[0], o[1], o[2], o[3]));
      __stcs(p + 1, make_uint4(o[4], o[5], o[6], o[7]));
    }
  }
}

}  // namespace sdk

extern "C" int sd_kv_write_launch(int n, int Hkv, int D, const void* k, long ld_k, long hs_k,
                                  const void* v, long ld_v, long hs_v, const int32_t* slots,
                                  void* k_cache, void* v_cache, long st_block, long st_tok,
                                  long st_head, float* k_scale, float* v_scale, int num_blocks,
                                  int log2_bs, int32_t* err, cudaStream_t stream) {
  sdk::KvWriteParams P;
  P.x[0] = (const uint16_t*)k;
  P.x[1] = (const uint16_t*)v;
  P.ld[0] = ld_k;
  P.ld[1] = ld_v;
  P.hs[0] = hs_k;
  P.hs[1] = hs_v;
  P.cache[0] = (uint8_t*)k_cache;
  P.cache[1] = (uint8_t*)v_cache;
  P.scale[0] = k_scale;
  P.scale[1] = v_scale;
  P.st_block = st_block;
  P.st_tok = st_tok;
  P.st_head = st_head;
  P.n = n;
  P.Hkv = Hkv;
  P.D = D;
  P.num_blocks = num_blocks;
  P.log2_bs = log2_bs;
  P.slots = slots;
  P.err = err;
  const int bs = 1 << log2_bs;
  const int team_warps = bs > 16 ? bs / 16 : 1;
  const int teams = (sdk::kWriteThreads / 32) / team_warps;
  const int gy = (2 * Hkv + teams - 1) / teams;
  // Few tokens: 8 a CTA, so that a step's runs spread over the SMs; many: 32, for the neighbouring
  // heads and tokens that a CTA then reads together. Steps of 6 or 8 tokens a request with 8 against
  // 32: 384 tokens 6.3 to 12.3 us, 2048 6.8 to 11.4, 4096 11.1 to 12.9, 8192 17.9 to 16.5; prompts:
  // 4096 tokens 7.9 to 7.3, 8192 12.9 to 11.3, 16384 22.6 to 18.7 (D = 64 and 128, 8 heads).
  P.chunk = (long)n * gy <= 8L * 152 * 8 ? 8 : 32;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((n + P.chunk - 1) / P.chunk), (unsigned)(gy < 65535 ? gy : 65535), 1);
  cfg.blockDim = dim3(sdk::kWriteThreads, 1, 1);
  cfg.dynamicSmemBytes = (size_t)P.chunk * bs * sizeof(int32_t);
  cfg.stream = stream;
  return cudaLaunchKernelEx(&cfg, sdk::kv_write_kernel, P) == cudaSuccess ? SD_OK : SD_E_LAUNCH;
}

extern "C" int sd_kv_read_launch(int B, int n, int Hkv, int D, const void* k_cache,
                                 const void* v_cache, long st_block, long st_tok, long st_head,
                                 const float* k_scale, const float* v_scale, int num_blocks,
                                 int log2_bs, const int32_t* table, int max_blocks,
                                 const int32_t* cu, const int32_t* first, void* k_out, void* v_out,
                                 long ld, long hs, int32_t* err, cudaStream_t stream) {
  sdk::KvReadParams P;
  P.c = sdk::KvCache{(const uint8_t*)k_cache, (const uint8_t*)v_cache, k_scale, v_scale,
                     st_block, st_tok, st_head, num_blocks, log2_bs, Hkv, D};
  P.B = B;
  P.n = n;
  P.max_blocks = max_blocks;
  P.table = table;
  P.cu = cu;
  P.first = first;
  P.out[0] = (uint16_t*)k_out;
  P.out[1] = (uint16_t*)v_out;
  P.ld = ld;
  P.hs = hs;
  P.err = err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((n + sdk::kReadRows - 1) / sdk::kReadRows), 1, 1);
  cfg.blockDim = dim3(sdk::kReadThreads, 1, 1);
  cfg.stream = stream;
  return cudaLaunchKernelEx(&cfg, sdk::kv_read_kernel, P) == cudaSuccess ? SD_OK : SD_E_LAUNCH;
}
