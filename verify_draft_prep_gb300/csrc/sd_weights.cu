// sd_weights.cu -- the attention weight that each cached token gets from a call's queries
// (sd_kv_weights), on the fifth-generation tensor cores.
//
// w[t] = sum over the query tokens i that count and the heads g of the group, of those that see t,
// e^(sm_scale q_ig . k_t - lse_ig), added to `decay` times what t had before (nothing for the call's
// own tokens).
//
// The sums of the softmax are an input, so nothing runs along a row: a tile's tokens stand in the 128
// lanes of the accumulator and the rows (a query token and one of the heads that share the KV head)
// in its columns, S^T = K Q^T, and every token's sum stays in the registers of the one thread that
// owns it. No maximum, no second product, no atomics, and the same call gives the same bits. Products are
// bf16: an e4m3 value is one exactly, and so is q, which then needs neither scales nor a second term; K
// is converted on its way to shared memory, where a byte waits for memory longer than for that.
//
// A unit is a pair of tiles (256 tokens) of one request and KV head; a chunk is up to 128 rows. Both
// tiles use a chunk of Q in shared memory, and one group of four warps turns the S of each into sums.
// Eight warps load: K (three units ahead through a ring in shared memory for heads of up to 64, else
// one ahead in registers, with one warp that has the units further on fetched into L2), and Q, which
// stays where a request has at most two chunks and else streams by, asynchronously copied, two chunks
// ahead. One thread issues the products.
//
// An exponential is the hardware's (off by two places) of an argument that is one fma of S, the scale and
// lse: off by 2^-24 of it, as lse itself is. 64 requests' numbers come out 5.0e-8 of their size from 64
// bits, plain fp32 ones 4.3e-8, a prompt's 1.8e-7 against 2.0e-7.
//
// What bounds it (pages of 16, 8 heads of K; shares of the active cycles, of one launch each):
//   - 64 requests of 6 slots, 64 heads of 64, 512 to 8192 tokens: 85 us against 22 of memory. Nothing is
//     full (issue slots 55%, memory 35%, exponentials 17%, tensor cores 9%): the loading warps' own chain,
//     some 450 instructions a unit each, is what the others wait for. K a unit ahead in registers: 95;
//     two units ahead in registers: 134 (spills).
//   - A prompt of 8192 tokens of 32 heads of 128: 362 us against 146 of products and 133 of exponentials.
//     Nothing is full either (exponentials and tensor cores 36% each, issue slots 45%): the summing warps,
//     two on a scheduler, each wait for their S with nothing on its way behind it. (With a quarter or an
//     eighth of the exponentials by a polynomial it took 519 and 480 us, without 437, when the loads took
//     more of the slots.)
//   - One token at 32000, 32 heads of 128: 19 us against 5: 7 units a CTA, each as long as its loads (issue
//     slots 35%, memory 18%); 26 with all of a unit's K in registers, some of which were spilled.
// S read 16 columns at a time with the next ones on their way: 64 requests 102 against 95 us, a prompt
// 502 against 437 (registers); three warps that fetch ahead, or 8 and 12 units: no change.

#include "sd_kv.cuh"
#include "sd_tc.cuh"

namespace sdk {

constexpr int kWTile = 128, kWPair = 2 * kWTile, kWRows = 128;
constexpr int kWThreads = 576;      // 8 warps sum, 8 load, one issues, one fetches ahead
constexpr int kWLoaders = 256;
constexpr int kWAhead = 5;  // units that are fetched ahead into L2
constexpr float kWLog2e = 1.4426950408889634f;

struct WeightsParams {
  KvCache c;
  int B, n, Hq, G, max_blocks, causal;
  unsigned long long g_magic;  // ceil(2^64 / G); 0 for G = 1
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

// LONG: requests of many chunks (prompts), whose Q streams by while K stays.
template <int DP, bool LONG>
struct WLayout {
  static constexpr int kTileBytes = kWTile * DP * 2;  // K of a tile, or Q of a chunk, as bf16
  static constexpr int kNK = LONG ? 1 : 2;            // pairs of tiles
  static constexpr int kNQ = LONG ? 4 : 2;            // chunks
  // Heads of up to 64 leave room for K's bytes on their way: a ring of units, which no thread holds in
  // registers.
  static constexpr int kRing = DP == 64 && !LONG ? 4 : 0;
  static constexpr int kRingUnit = kWPair * (DP + 16);  // bytes, scale, number so far and its place
  static constexpr int kK = 0;
  static constexpr int kQ = kK + 2 * kNK * kTileBytes;
  static constexpr int kStage = kQ + kNQ * kTileBytes;
  static constexpr int kMisc = kStage + kRing * kRingUnit;
};

struct WMisc {
  uint64_t k_full[2], k_empty[2], q_full[4], q_empty[4];
  uint64_t s_full[2][2], s_empty[2][2];  // [tile of the pair][buffer]
  float lse2[4][kWRows];                 // -lse log2(e) of the rows of a chunk of Q
  int lim[4][kWRows];                    // tokens that they see
  float k_scale[2][kWPair];              // of a pair's tokens, times sm_scale log2(e)
  float before[2][kWPair];               // what they have so far
  long at[2][kWPair];                    // where their number lies; -1: nowhere
  long long warp_sum[kWThreads / 32];
  int start_r;
  long long start_in;
  uint32_t tmem;
  int gave_up;
  int loaded;  // units that are on their way to shared memory
};

struct WRequest {
  int tok0, rows, len, off;  // rows: those that count
};

__device__ __forceinline__ int w_token(const WeightsParams& P, int row) {
  return P.g_magic ? (int)__umul64hi((unsigned long long)row, P.g_magic) : row;
}
__device__ __forceinline__ long w_covered(const WeightsParams& P) {
  return min((long)P.max_blocks << P.c.log2_bs, 2147483648L - 2 * kWPair);
}
__device__ __forceinline__ WRequest w_request(const WeightsParams& P, int r) {
  WRequest q;
  const int a = P.cu[r], b = P.cu[r + 1], ctx = P.ctx[r];
  const int lo = min(max(a, 0), P.n), hi = min(max(b, lo), P.n);
  const int n_q = hi - lo;
  q.tok0 = lo;
  q.rows = (P.live ? min(max(P.live[r], 0), n_q) : n_q) * P.G;
  q.len = ctx < 0 ? 0 : (int)min((long)ctx, w_covered(P));
  q.off = (int)max((long)ctx - n_q, -2147483647L);
  return q;
}
__device__ __forceinline__ bool w_bad(const WeightsParams& P, int r) {
  const int a = P.cu[r], b = P.cu[r + 1], ctx = P.ctx[r];
  const bool bad = a < 0 || b < a || b > P.n || ctx < 0 || ctx > w_covered(P);
  return bad || (P.live && (P.live[r] < 0 || P.live[r] > b - a));
}
__device__ __forceinline__ int w_sees(const WeightsParams& P, const WRequest& q, int row) {
  if (!P.causal) return q.len;
  return (int)max(0L, min((long)q.len, (long)q.off + w_token(P, row) + 1));
}

// A pair of tiles of one request and KV head, and the chunks of rows that see any of its tokens.
struct WUnit {
  WRequest q;
  int r, h, pair, first, chunks;
};
// A chunk of Q stays for the next unit where the request has at most two of them.
__device__ __forceinline__ bool w_stays(const WUnit& a, const WUnit& b, bool there) {
  return there && a.chunks <= 2 && a.r == b.r && a.h == b.h;
}

// A CTA's units in their order. All units of a request lie one behind another; `spread`: pairs
// outermost and every CTA takes one of each gridDim.x units, forwards and backwards in turn, so that a
// prompt's units, which get cheaper along the context, even out; else heads outermost and every CTA
// takes a stretch, so that it stays with a request's Q.
template <bool SPREAD>
struct WSchedule {
  long long at, end;  // place on the line
  int pairs, round;

  __device__ __forceinline__ void place(const WeightsParams& P, WUnit& u, int h, int pair) const {
    u.h = h;
    u.pair = pair;
    u.first = 0;
    if (P.causal && u.chunks > 2)
      u.first = (int)min((long)u.chunks, max(0L, (long)pair * kWPair - u.q.off) * P.G / kWRows);
  }
  __device__ __forceinline__ void request(const WeightsParams& P, WUnit& u, int r) {
    u.r = r;
    u.q = w_request(P, r);
    u.chunks = (u.q.rows + kWRows - 1) / kWRows;
    pairs = (u.q.len + kWPair - 1) / kWPair;
  }
  // `in` places behind the first unit of u's request.
  __device__ __forceinline__ void seek(const WeightsParams& P, WUnit& u, long long in) {
    for (;;) {
      const long long units = (long long)pairs * P.c.Hkv;
      if (in < units) break;
      in -= units;
      request(P, u, u.r + 1);
    }
    const int by = SPREAD ? P.c.Hkv : pairs;
    const int o = (int)(in / by), i = (int)(in - (long long)o * by);
    place(P, u, SPREAD ? i : o, SPREAD ? o : i);
  }
  __device__ __forceinline__ WUnit begin(const WeightsParams& P, long long from, long long to, int r,
                                         long long in) {
    at = from;
    end = to;
    round = pairs = 0;
    WUnit u = {};
    if (from < to) {
      request(P, u, r);
      seek(P, u, in);
    }
    return u;
  }
  // On to the next unit; false: there is none.
  __device__ __forceinline__ bool next(const WeightsParams& P, WUnit& u) {
    if (SPREAD) {
      const int n = gridDim.x, b = blockIdx.x;
      const int by = round++ & 1 ? 2 * b + 1 : 2 * (n - 1 - b) + 1;
      at += by;
      if (at >= end) return false;
      seek(P, u, (long long)u.pair * P.c.Hkv + u.h + by);
      return true;
    }
    if (++at >= end) return false;
    if (u.pair + 1 < pairs) {
      place(P, u, u.h, u.pair + 1);
    } else if (u.h + 1 < P.c.Hkv) {
      place(P, u, u.h + 1, 0);
    } else {
      do request(P, u, u.r + 1);
      while (pairs == 0);
      place(P, u, 0, 0);
    }
    return true;
  }
};

// 16 e4m3 bytes as bf16 (two 16-byte parts), exactly.
__device__ __forceinline__ void to_bf16(const uint4& v, uint4& lo, uint4& hi) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = e4m3x2_to_f32((uint16_t)w[i]), b = e4m3x2_to_f32((uint16_t)(w[i] >> 16));
    // (the lower halves of these fp32 are zero)
    o[2 * i] = __byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x7632);
    o[2 * i + 1] = __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x7632);
  }
  lo = make_uint4(o[0], o[1], o[2], o[3]);
  hi = make_uint4(o[4], o[5], o[6], o[7]);
}

__device__ __forceinline__ float w_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float2 w_fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(*reinterpret_cast<unsigned long long*>(&d))
      : "l"(*reinterpret_cast<const unsigned long long*>(&a)),
        "l"(*reinterpret_cast<const unsigned long long*>(&b)),
        "l"(*reinterpret_cast<const unsigned long long*>(&c)));
  return d;
}
__device__ __forceinline__ float2 w_add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(*reinterpret_cast<unsigned long long*>(&d))
      : "l"(*reinterpret_cast<const unsigned long long*>(&a)),
        "l"(*reinterpret_cast<const unsigned long long*>(&b)));
  return d;
}

__device__ __forceinline__ void w_copy4(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(there ? 4 : 0)
               : "memory");
}
__device__ __forceinline__ void w_copy16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(there ? 16 : 0)
               : "memory");
}

template <int DP, bool LONG>
__global__ void __launch_bounds__(kWThreads, 1) weights_kernel(const WeightsParams P) {
  using L = WLayout<DP, LONG>;
  extern __shared__ unsigned char s_raw[];
  unsigned char* smem = s_raw + ((1024 - (smem_u32(s_raw) & 1023)) & 1023);
  WMisc& m = *reinterpret_cast<WMisc*>(smem + L::kMisc);
  const KvCache& c = P.c;
  const uint32_t base = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* gave_up = &m.gave_up;
  const int bs = 1 << c.log2_bs;

  if (tid < 4) {
    mbar_init(smem_u32(&m.q_full[tid]), 8);
    mbar_init(smem_u32(&m.q_empty[tid]), 9);
    mbar_init(smem_u32(&m.s_full[tid >> 1][tid & 1]), 1);
    mbar_init(smem_u32(&m.s_empty[tid >> 1][tid & 1]), 4);
    if (tid < 2) {
      mbar_init(smem_u32(&m.k_full[tid]), 8);
      mbar_init(smem_u32(&m.k_empty[tid]), 9);
    }
    m.gave_up = 0;
    m.loaded = 0;
    m.start_r = P.B;
  }
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  if (warp == 16) tmem_alloc(smem_u32(&m.tmem), 512);
  // What comes before this call on its stream may still be running up to here.
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // ---- this CTA's place on the line of units ----
  const int per = (P.B + kWThreads - 1) / kWThreads;
  const int r0 = min(P.B, tid * per), r1 = min(P.B, r0 + per);
  long long mine = 0;
  bool bad = false;
  for (int r = r0; r < r1; ++r) {
    mine += (long long)((w_request(P, r).len + kWPair - 1) / kWPair) * c.Hkv;
    if (blockIdx.x == 0) bad |= w_bad(P, r);
  }
  if (bad) raise_err(P.err, SD_ERR_KV_RANGE);
  long long before = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += x;
  }
  if (lane == 31) m.warp_sum[warp] = before;
  __syncthreads();
  long long total = 0;
  before -= mine;
  for (int w = 0; w < kWThreads / 32; ++w) {
    if (w < warp) before += m.warp_sum[w];
    total += m.warp_sum[w];
  }
  const long long share = (total + gridDim.x - 1) / gridDim.x;
  const long long g0 = LONG ? blockIdx.x : min(total, share * blockIdx.x);
  const long long g1 = LONG ? total : min(total, g0 + share);
  if (g0 < g1 && before <= g0 && g0 < before + mine) {
    long long in = g0 - before;
    int r = r0;
    for (; r < r1; ++r) {
      const long long u = (long long)((w_request(P, r).len + kWPair - 1) / kWPair) * c.Hkv;
      if (in < u) break;
      in -= u;
    }
    m.start_r = r;
    m.start_in = in;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = m.tmem;
  WSchedule<LONG> line;
  WUnit s = line.begin(P, g0, g1, m.start_r, m.start_in);
  bool some = g0 < g1;

  if (warp >= 8 && warp < 16) {
    // ---- loads ----
    const int t = tid - kWLoaders, lw = t >> 5;
    constexpr int kParts = DP / 16, kPerPass = 32 / kParts;  // parts of a token; tokens of a pass
    constexpr int kPasses = 32 / kPerPass;                   // of a warp's 32 tokens: 8 or 4
    const int part = lane % kParts, sub = lane / kParts;
    constexpr int kHeld = 4;  // passes whose bytes are in registers at a time
    uint4 x[kHeld];
    float ks = 0.f, was = 0.f;
    long where = -1, src = -1;
    int page_next = -1;
    volatile int* loaded = &m.loaded;
    auto page_of = [&](const WUnit& u) {
      const int tok = u.pair * kWPair + t;
      return tok < u.q.len ? __ldg(P.table + (long)u.r * P.max_blocks + (tok >> c.log2_bs)) : -2;
    };
    auto bytes = [&](int first) {  // of kHeld passes
#pragma unroll
      for (int i = 0; i < kHeld; ++i) {
        const long from = __shfl_sync(0xffffffffu, src, (first + i) * kPerPass + sub);
        x[i] = make_uint4(0, 0, 0, 0);
        if (from >= 0 && part * 16 < c.D) x[i] = ld_stream_u4(c.k + from + part * 16);
      }
    };
    auto fetch = [&](const WUnit& u, int page) {  // this warp's tokens of a unit
      const int tok = u.pair * kWPair + t;
      ks = 0.f;
      was = 0.f;
      where = src = -1;
      if ((unsigned)page < (unsigned)c.num_blocks) {
        const long slot = (long)page * c.Hkv + u.h;
        ks = __ldg(c.k_scale + slot);
        where = slot * bs + (tok & (bs - 1));
        if (P.before && tok < u.q.off) was = P.before[where];
        src = page * c.st_block + (tok & (bs - 1)) * c.st_tok + u.h * c.st_head;
      } else if (page != -2) {
        raise_err(P.err, SD_ERR_KV_RANGE);
      }
      bytes(0);
    };
    WUnit ahead = s;
    bool more = some;
    // The ring: every thread copies for itself and waits for its own copies alone.
    constexpr int kRing = L::kRing > 0 ? L::kRing : 1;
    WSchedule<LONG> far = line;
    auto stage_of = [&](int u) { return (uint32_t)(L::kStage + u % kRing * L::kRingUnit); };
    auto issue = [&](int u) {  // unit number u, which is `ahead`
      if (more) {
        const uint32_t st = base + stage_of(u);
        const int tok = ahead.pair * kWPair + t, page = page_next;
        const bool is = (unsigned)page < (unsigned)c.num_blocks;
        if (!is && page != -2) raise_err(P.err, SD_ERR_KV_RANGE);
        const long slot = is ? (long)page * c.Hkv + ahead.h : 0;
        const long to = is ? slot * bs + (tok & (bs - 1)) : -1;
        const long from = is ? page * c.st_block + (tok & (bs - 1)) * c.st_tok + ahead.h * c.st_head : -1;
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
          const long at = __shfl_sync(0xffffffffu, from, i * kPerPass + sub);
          const bool there = at >= 0 && part * 16 < c.D;
          w_copy16(st + (i * kWLoaders + t) * 16, c.k + (there ? at + part * 16 : 0), there);
        }
        const uint32_t meta = st + kWPair * DP + t * 4;
        w_copy4(meta, c.k_scale + slot, is);
        const bool old = is && P.before && tok < ahead.q.off;
        w_copy4(meta + kWPair * 4, old ? P.before + to : c.k_scale, old);
        *reinterpret_cast<long*>(smem + stage_of(u) + kWPair * (DP + 8) + t * 8) = to;
        more = far.next(P, ahead);
        if (more) page_next = page_of(ahead);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if (L::kRing > 0) {
      if (more) page_next = page_of(ahead);
      for (int u = 0; u + 1 < kRing; ++u) issue(u);
    } else if (more) {
      fetch(s, page_of(s));
      more = line.next(P, ahead);
      if (more) page_next = page_of(ahead);
    }
    int unit = 0, loads = 0;
    bool ok = true, have_q = false;
    while (some && ok) {
      const int kb = unit % L::kNK;
      if (L::kRing > 0) {
        issue(unit + kRing - 1);
        asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
        const unsigned char* st = smem + stage_of(unit);
#pragma unroll
        for (int i = 0; i < kPasses; ++i)
          x[i % kHeld] = *reinterpret_cast<const uint4*>(st + (i * kWLoaders + t) * 16);
        ks = *reinterpret_cast<const float*>(st + kWPair * DP + t * 4);
        was = *reinterpret_cast<const float*>(st + kWPair * (DP + 4) + t * 4);
        where = *reinterpret_cast<const long*>(st + kWPair * (DP + 8) + t * 8);
      }
      ok = mbar_wait_warp(smem_u32(&m.k_empty[kb]), ((unit / L::kNK) & 1) ^ 1, gave_up);
      if (!ok) break;
      // K of this unit, which is in registers
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        // (heads of 128: the second half is in L2 by now)
        if (L::kRing == 0 && i > 0 && i % kHeld == 0) bytes(i);
        const int tok = lw * 32 + i * kPerPass + sub;
        const float f = __shfl_sync(0xffffffffu, ks, i * kPerPass + sub);
        uint4 lo, hi;
        to_bf16(f == 0.f ? make_uint4(0, 0, 0, 0) : x[i % kHeld], lo, hi);  // a scale of 0: zeros
        const int row = tok & (kWTile - 1), ch = (2 * part) & 7;
        unsigned char* at = smem + L::kK + (kb * 2 + (tok >> 7)) * L::kTileBytes +
                            (part >> 2) * (kWTile * 128) + row * 128;
        *reinterpret_cast<uint4*>(at + ((ch ^ (row & 7)) << 4)) = lo;
        *reinterpret_cast<uint4*>(at + (((ch + 1) ^ (row & 7)) << 4)) = hi;
      }
      m.k_scale[kb][t] = ks * P.scale;
      m.before[kb][t] = was;
      m.at[kb][t] = where;
      fence_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&m.k_full[kb]));
      // the next unit's K on its way
      WUnit after = ahead;
      bool next_there = more;
      if (L::kRing > 0) {
        after = s;
        next_there = line.next(P, after);
      } else if (more) {
        fetch(ahead, page_next);
        more = line.next(P, ahead);
        if (more) page_next = page_of(ahead);
      }
      if (t == 0) *loaded = unit + 1;
      // Q, chunk by chunk
      if (LONG) {
        // by asynchronous copies, two chunks on their way behind the one that is waited for
        constexpr int kLanes = DP / 8, kRowsPass = kWLoaders / kLanes;
        const int d8 = t % kLanes;
        auto of_row = [&](int ch, float& l2, int& lim) {
          l2 = -INFINITY;
          lim = 0;
          const int row = ch * kWRows + t;
          if (t < kWRows && row < s.q.rows && ch < s.chunks) {
            const int tk = w_token(P, row);
            l2 = __ldg(P.lse + (long)(s.q.tok0 + tk) * P.Hq + s.h * P.G + row - tk * P.G) * -kWLog2e;
            lim = w_sees(P, s.q, row);
          }
        };
        auto there = [&](int load) {
          fence_async_shared();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&m.q_full[load % L::kNQ]));
        };
        float l2;
        int lim;
        of_row(s.first, l2, lim);
        for (int ch = s.first; ok && ch < s.chunks; ++ch, ++loads) {
          const int qb = loads % L::kNQ;
          ok = mbar_wait_warp(smem_u32(&m.q_empty[qb]), ((loads / L::kNQ) & 1) ^ 1, gave_up);
          if (!ok) break;
          // a warp's 16 rows: a lane finds one, all lanes copy
          long mine = -1;
          const int at0 = (t >> 5) * (32 / kLanes) + (lane & 15) % (32 / kLanes) +
                          (lane & 15) / (32 / kLanes) * kRowsPass;
          if (lane < 16 && ch * kWRows + at0 < s.q.rows) {
            const int row = ch * kWRows + at0, tk = w_token(P, row);
            mine = (long)(s.q.tok0 + tk) * P.ld_q + (long)(s.h * P.G + row - tk * P.G) * P.hs_q;
          }
#pragma unroll
          for (int i = 0; i < DP / 16; ++i) {
            const long from = __shfl_sync(0xffffffffu, mine, i * (32 / kLanes) + lane / kLanes);
            const int at = i * kRowsPass + t / kLanes;
            const bool is = from >= 0 && d8 * 8 < c.D;
            w_copy16(base + L::kQ + qb * L::kTileBytes + (d8 >> 3) * (kWRows * 128) + at * 128 +
                         (((d8 & 7) ^ (at & 7)) << 4),
                     P.q + (is ? from + d8 * 8 : 0), is);
          }
          asm volatile("cp.async.commit_group;" ::: "memory");
          if (t < kWRows) {
            m.lse2[qb][t] = l2;
            m.lim[qb][t] = lim;
          }
          of_row(ch + 1, l2, lim);
          if (ch - s.first >= 2) {
            asm volatile("cp.async.wait_group 2;" ::: "memory");
            there(loads - 2);
          }
        }
        if (ok && s.chunks - s.first >= 2) {
          asm volatile("cp.async.wait_group 1;" ::: "memory");
          there(loads - 2);
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        if (ok && s.chunks > s.first) there(loads - 1);
      } else if (!have_q) {
        for (int ch = s.first; ok && ch < s.chunks; ++ch, ++loads) {
          const int qb = loads & 1;
          const int row0 = ch * kWRows;
          constexpr int kLanes = DP / 8, kRowsPass = kWLoaders / kLanes;
          const int d8 = t % kLanes;
          uint4 y[4];
          auto q_rows = [&](int i0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int row = row0 + (i0 + i) * kRowsPass + t / kLanes;
              y[i] = make_uint4(0, 0, 0, 0);
              if (row < s.q.rows && d8 * 8 < c.D) {
                const int tk = w_token(P, row);
                y[i] = __ldg(reinterpret_cast<const uint4*>(
                    P.q + (long)(s.q.tok0 + tk) * P.ld_q +
                    (long)(s.h * P.G + row - tk * P.G) * P.hs_q + d8 * 8));
              }
            }
          };
          q_rows(0);
          float l2 = -INFINITY;
          int lim = 0;
          if (t < kWRows && row0 + t < s.q.rows) {
            const int row = row0 + t, tk = w_token(P, row);
            l2 = __ldg(P.lse + (long)(s.q.tok0 + tk) * P.Hq + s.h * P.G + row - tk * P.G) * -kWLog2e;
            lim = w_sees(P, s.q, row);
          }
          ok = mbar_wait_warp(smem_u32(&m.q_empty[qb]), ((loads >> 1) & 1) ^ 1, gave_up);
          if (!ok) break;
#pragma unroll
          for (int i0 = 0; i0 < DP / 16; i0 += 4) {
            if (i0) q_rows(i0);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int row = (i0 + i) * kRowsPass + t / kLanes;
              *reinterpret_cast<uint4*>(smem + L::kQ + qb * L::kTileBytes +
                                        (d8 >> 3) * (kWRows * 128) + row * 128 +
                                        (((d8 & 7) ^ (row & 7)) << 4)) = y[i];
            }
          }
          if (t < kWRows) {
            m.lse2[qb][t] = l2;
            m.lim[qb][t] = lim;
          }
          fence_async_shared();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&m.q_full[qb]));
        }
      }
      have_q = !LONG && w_stays(s, after, next_there);
      s = after;
      some = next_there;
      ++unit;
    }
  } else if (warp == 16) {
    // ---- products ----
    constexpr uint32_t hi = desc_hi<128>();
    const bool lead = elect_one();
    const uint32_t k_lo = desc_lo<128>(base + L::kK), q_lo = desc_lo<128>(base + L::kQ);
    int unit = 0, loads = 0, jobs[2] = {0, 0};
    bool ok = true;
    while (some && ok) {
      const int kb = unit % L::kNK;
      WUnit after = s;
      const bool there = line.next(P, after);
      const bool keep = !LONG && w_stays(s, after, there);
      ok = mbar_wait_warp(smem_u32(&m.k_full[kb]), (unit / L::kNK) & 1, gave_up);
      const bool two = (long)s.pair * kWPair + kWTile < s.q.len;
      for (int ch = s.first; ok && ch < s.chunks; ++ch) {
        const int load = loads + ch - s.first, qb = load % L::kNQ;
        ok = mbar_wait_warp(smem_u32(&m.q_full[qb]), (load / L::kNQ) & 1, gave_up);
        const int cols = min(kWRows, (s.q.rows - ch * kWRows + 31) & ~31);
        const uint32_t idesc = mma_desc_bf16(cols);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (!ok || (x && !two)) continue;
          const int sb = jobs[x] & 1;
          ok = mbar_wait_warp(smem_u32(&m.s_empty[x][sb]), ((jobs[x] >> 1) & 1) ^ 1, gave_up);
          if (!ok) continue;
          ++jobs[x];
          tc_fence_after();
          if (lead) {
            const uint32_t d = tmem + (x * 2 + sb) * kWRows;
            const uint32_t a = k_lo + (kb * 2 + x) * (L::kTileBytes / 16),
                           b = q_lo + qb * (L::kTileBytes / 16);
#pragma unroll
            for (int kk = 0; kk < DP / 16; ++kk) {
              const uint32_t o = (kk >> 2) * (kWTile * 128 / 16) + (kk & 3) * 2;
              mma_ss_bf16<hi>(d, a + o, b + o, idesc, kk > 0);
            }
            mma_commit(smem_u32(&m.s_full[x][sb]));
          }
        }
        if (ok && lead && !keep) mma_commit(smem_u32(&m.q_empty[qb]));
      }
      if (ok && lead) mma_commit(smem_u32(&m.k_empty[kb]));
      if (!keep) loads += s.chunks - s.first;
      s = after;
      some = there;
      ++unit;
      __syncwarp();
    }
    __syncwarp();
  } else if (warp == 17) {
    // ---- K of the units to come into L2: a unit's registers alone do not keep memory busy ----
    if (!LONG && L::kRing == 0) {
      volatile int* loaded = &m.loaded;
      const long long t0 = clock64();
      for (int unit = 0; some; ++unit) {
        int page[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int tok = s.pair * kWPair + i * 32 + lane;
          page[i] = tok < s.q.len ? __ldg(P.table + (long)s.r * P.max_blocks + (tok >> c.log2_bs)) : -1;
        }
        while (unit - *loaded > kWAhead && !*gave_up && clock64() - t0 < kWaitClocks) __nanosleep(100);
        if (*gave_up || clock64() - t0 >= kWaitClocks) break;
        if (unit > *loaded) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if ((unsigned)page[i] >= (unsigned)c.num_blocks) continue;
            const int tok = s.pair * kWPair + i * 32 + lane;
            const uint8_t* at = c.k + page[i] * c.st_block + (tok & (bs - 1)) * c.st_tok + s.h * c.st_head;
            asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
          }
        }
        __syncwarp();
        some = line.next(P, s);
      }
    }
  } else {
    // ---- sums: group x has tile x of the pair, a token a lane ----
    const int x = warp >> 2, wt = tid & (kWTile - 1);
    const uint32_t tS = tmem + x * 2 * kWRows + ((uint32_t)(warp & 3) << 21);
    int unit = 0, loads = 0, jobs = 0;
    bool ok = true;
    while (some && ok) {
      const int kb = unit % L::kNK;
      WUnit after = s;
      const bool there = line.next(P, after);
      const bool keep = !LONG && w_stays(s, after, there);
      ok = mbar_wait_warp(smem_u32(&m.k_full[kb]), (unit / L::kNK) & 1, gave_up);
      const int t0 = s.pair * kWPair + x * kWTile, tok = t0 + wt;
      const bool mine_any = t0 < s.q.len;
      const float f = m.k_scale[kb][x * kWTile + wt];
      const float2 f2 = make_float2(f, f);
      float sum = 0.f, rest = 0.f;  // (compensated from chunk to chunk)
      for (int ch = s.first; ok && ch < s.chunks; ++ch) {
        const int load = loads + ch - s.first, qb = load % L::kNQ;
        ok = mbar_wait_warp(smem_u32(&m.q_full[qb]), (load / L::kNQ) & 1, gave_up);
        if (!ok) break;
        if (mine_any) {
          const int sb = jobs & 1;
          ok = mbar_wait_warp(smem_u32(&m.s_full[x][sb]), (jobs >> 1) & 1, gave_up);
          if (!ok) break;
          ++jobs;
          tc_fence_after();
          const int cols = min(kWRows, (s.q.rows - ch * kWRows + 31) & ~31);
          // rows see more along a chunk; the first sees the whole tile, or some tokens are masked
          const bool masked = m.lim[qb][0] < t0 + kWTile;
          const uint32_t tC = tS + sb * kWRows;
          float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          // 32 columns at a time
          auto add = [&](const uint32_t (&v)[32], int c0) {
            const float4* l4 = reinterpret_cast<const float4*>(&m.lse2[qb][c0]);
            if (!masked) {
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float4 l = l4[i];
                const float2 a = w_fma2(make_float2(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1])),
                                        f2, make_float2(l.x, l.y));
                const float2 b = w_fma2(
                    make_float2(__uint_as_float(v[4 * i + 2]), __uint_as_float(v[4 * i + 3])), f2,
                    make_float2(l.z, l.w));
                acc[0] = w_add2(acc[0], make_float2(w_ex2(a.x), w_ex2(a.y)));
                acc[1] = w_add2(acc[1], make_float2(w_ex2(b.x), w_ex2(b.y)));
              }
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const float e = w_ex2(fmaf(__uint_as_float(v[i]), f, m.lse2[qb][c0 + i]));
                acc[i & 1].x += tok < m.lim[qb][c0 + i] ? e : 0.f;
              }
            }
          };
          for (int c0 = 0; c0 < cols; c0 += 32) {
            uint32_t v[32];
            tmem_ld32(tC + c0, v);
            tmem_wait_ld();
            add(v, c0);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&m.s_empty[x][sb]));
          const float part = (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
          const float y = part - rest, z = sum + y;
          rest = (z - sum) - y;
          sum = z;
        }
        __syncwarp();
        if (lane == 0 && !keep) mbar_arrive(smem_u32(&m.q_empty[qb]));
      }
      if (ok) {
        const long at = m.at[kb][x * kWTile + wt];
        if (at >= 0) P.weights[at] = fmaf(P.decay, m.before[kb][x * kWTile + wt], sum);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&m.k_empty[kb]));
      if (!keep) loads += s.chunks - s.first;
      s = after;
      some = there;
      ++unit;
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (m.gave_up) {
    // a wait ran out: the products in flight get some milliseconds before the memory is given up
    if (tid == 0) raise_err(P.err, SD_ERR_WAIT);
    const long long t = clock64();
    while (clock64() - t < 20000000LL) __nanosleep(1000);
    __syncthreads();
  }
  tc_fence_after();
  if (warp == 16) tmem_free(tmem, 512);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <int DP, bool LONG>
static int launch_weights(const WeightsParams& P, cudaStream_t stream) {
  constexpr int smem = WLayout<DP, LONG>::kMisc + (int)sizeof(WMisc) + 1024;
  static_assert(smem <= 227 * 1024, "shared memory of one CTA");
  static std::atomic<bool> set[kMostDevices];  // true only once the attribute is in force
  int dev = 0;
  const int sms = device_sms(dev);
  if (sms == 0) return SD_E_DEVICE;
  if (!set[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(weights_kernel<DP, LONG>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             smem) != cudaSuccess)
      return SD_E_LAUNCH;
    set[dev].store(true, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)sms, 1, 1);
  cfg.blockDim = dim3(kWThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, weights_kernel<DP, LONG>, P) == cudaSuccess ? SD_OK : SD_E_LAUNCH;
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
  P.g_magic = P.G > 1 ? ~0ull / (unsigned)P.G + 1 : 0;
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
  P.scale = sm_scale * sdk::kWLog2e;
  P.decay = decay;
  P.before = before;
  P.weights = weights;
  P.err = err;
  // Prompts of many chunks, by the rows of the longest request that the caller expects. The kernel for few
  // against the one for many, in us, without a context and behind one of 8000 tokens (one request, 8 heads
  // of K):
  //   heads of 128:  1024 rows 20 to 20 (4 requests), 2048 32.0 to 30.9 and 56.5 to 56.3, 4096 55.4 to 52.8
  //     and 103 to 100, 8192 102 to 97 and 291 to 188, 32768 747 to 360; 16 requests of 2048 rows 48 to 50,
  //     4 of 2048 behind 4000 tokens 106 to 109.
  //   heads of 64:   2048 rows 27.9 to 29.9 and 49 to 54, 4096 49 to 52 and 91 to 97, 8192 90 to 95 and
  //     257 to 183 (4 requests 166 to 133, 16 233 to 256), 16384 173 to 181 and 506 to 357, 32768 661 to
  //     353; 64 requests of 48 rows 80 to 201.
  // (Where every CTA has one unit at most the two differ by their loops alone; with more the units of a
  // prompt are uneven, which the one for many spreads.)
  if ((long)max_q * P.G >= (D <= 64 ? 8192 : 4096))
    return D <= 64 ? sdk::launch_weights<64, true>(P, stream)
                   : sdk::launch_weights<128, true>(P, stream);
  return D <= 64 ? sdk::launch_weights<64, false>(P, stream)
                 : sdk::launch_weights<128, false>(P, stream);
}
