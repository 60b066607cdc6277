// sd_attend.cu -- attention over the paged 8-bit cache (sd_kv_attend), on the fifth-generation
// tensor cores.
//
// Query token i of request r stands at position ctx_lens[r] - n_q + i and sees every token up to
// its own position (causal) or all of them. With S = sm_scale q k, M the running maximum and L
// the running sum of the exponentials: O = sum e^(S - M) v / L, lse = M + ln L.
//
// The cache's bytes go to the tensor cores as they are, without being converted: an e4m3 value has
// 4 significant bits and bf16 has 8, so q is split into two e4m3 terms, q = q1 + q2 (after a power
// of two per row brings its largest magnitude to [224, 448]; exact but for values below 2^-17 of
// that), and so is each weight P = P1 + P2 (P at most 448 there, too). Two e4m3 products take the
// time of one bf16 product, and K and V cost half the shared memory and no instructions. A page's
// scales enter as numbers per 8 columns of S: with y = log2(e) S + log2(v_scale),
//   P = 2^(y - M + 8),  O = sum P v_byte,  L = sum P / v_scale,
// M the running maximum of y, so that one exponential serves both sums.
//
// A unit is one request's 128 (or 256) rows of one KV head; a row is a query token and one of the
// Hq / Hkv heads that share the KV head. All units' tiles of 128 tokens form one line, which the
// CTAs (one per SM) divide evenly, whatever the lengths of the requests: a unit that several CTAs
// share leaves its parts in the workspace and attend_join_kernel joins them in a fixed order.
// Within a CTA: warp 0 loads pages (TMA), warp 1 issues the products, warp 2 fetches scales, two
// groups of four warps turn S into P, one row a thread. The groups are two streams that keep
// the tensor cores busy in turn: with few rows they take alternate tiles of the same rows (and
// the accumulators are joined at the unit's end), with many they take 128 rows each of the same
// tiles, which halves the traffic of K and V.

#include "sd_kv.cuh"
#include "sd_tc.cuh"

namespace sdk {

constexpr int kTile = 128;                 // tokens of a tile, rows of a stream
constexpr int kAttThreads = 384;
constexpr int kMaxCtas = 160;
constexpr int kScaleSlots = 16;            // tiles of scales in flight
// A page whose V scale is 0 holds zeros: its tokens weigh in L only. They are given a scale below
// that of any page with values, so that those keep P's full precision.
constexpr float kZeroLog2 = -60.f, kZeroInv = 1152921504606846976.f;
constexpr float kLog2eF = 1.4426950408889634f, kLn2F = 0.6931471805599453f;

struct AttendParams {
  KvCache c;
  int B, n, Hq, G, max_blocks, causal, min_share;
  const uint16_t* q;
  long ld_q, hs_q;
  const int32_t* table;
  const int32_t* ctx;
  const int32_t* cu;
  float scale;  // sm_scale * log2(e)
  uint16_t* out;
  long ld_out, hs_out;
  float* lse;
  unsigned char* ws;
  int32_t* err;
};

// One unit's rows as the joining kernel needs them; a CTA leaves one for the unit that it begins
// and does not end.
struct JoinDesc {
  int pieces, tok0, head, row0, rows;
  int pad[3];
};

template <int DP, int NS>
struct AttLayout {
  // NS: Q tiles of a unit (1: the streams share one, 2: one each)
  static constexpr int kRows = NS * kTile;
  static constexpr int kQBytes = kTile * DP;        // one term of one Q tile
  static constexpr int kTileBytes = kTile * DP;     // K or V of one tile
  static constexpr int kStages = DP == 64 ? 8 : (NS == 1 ? 5 : 4);
  static constexpr int kQ = 0;
  static constexpr int kK = kQ + NS * 2 * kQBytes;
  static constexpr int kV = kK + kStages * kTileBytes;
  static constexpr int kScales = kV + kStages * kTileBytes;
  static constexpr int kMisc = kScales + kScaleSlots * 16 * 16;
  static constexpr long kSlotFloats = (long)kRows * DP + kRows;
};

struct AttMisc {
  uint64_t k_full[8], k_empty[8], v_full[8], v_empty[8];
  uint64_t s_full[2], p_full[2], o_done[2], q_full[2], q_empty[2];
  uint64_t sc_full[kScaleSlots], sc_empty[kScaleSlots];
  int sc_zero[kScaleSlots];   // bit e: entry e's V scale is zero
  float row_scale[2 * kTile];
  float2 ml[2][kTile];        // (M, L) of both streams
  int nan_first[2][128];      // first token with a NaN in dimension d of V, of a masked tile
  int nan_any[2];
  long long start[2];         // of the schedule
  int start_item[3];
  long long warp_sum[kAttThreads / 32];
  uint32_t tmem;
  int gave_up;
};

struct Request {
  int tok0, n_q, rows, len, off;
};

__device__ __forceinline__ Request request_of(const AttendParams& P, int r) {
  Request q;
  const int a = __ldg(P.cu + r), b = __ldg(P.cu + r + 1);
  const int lo = min(max(a, 0), P.n), hi = min(max(b, lo), P.n);
  q.tok0 = lo;
  q.n_q = hi - lo;
  q.rows = q.n_q * P.G;
  const int ctx = __ldg(P.ctx + r);
  const long cover = (long)P.max_blocks << P.c.log2_bs;
  q.len = ctx < 0 ? 0 : (int)min((long)ctx, cover);
  q.off = (int)max((long)ctx - q.n_q, -2147483647L);
  return q;
}

__device__ __forceinline__ bool request_bad(const AttendParams& P, int r) {
  const int a = P.cu[r], b = P.cu[r + 1], ctx = P.ctx[r];
  return a < 0 || b < a || b > P.n || ctx < 0 || ctx > ((long)P.max_blocks << P.c.log2_bs);
}

// Tokens that a row sees.
__device__ __forceinline__ int seen_by(const AttendParams& P, const Request& q, int row) {
  if (!P.causal) return q.len;
  const long t = (long)q.off + row / P.G + 1;
  return (int)max(0L, min((long)q.len, t));
}
// Tiles that rows up to `row` need; a row that sees nothing has one, in which all is masked.
__device__ __forceinline__ int tiles_for(const AttendParams& P, const Request& q, int row) {
  return max(1, (int)(((long)seen_by(P, q, row) + kTile - 1) / kTile));
}

// A CTA's part [a, b) of a unit's n tiles.
struct Segment {
  Request q;
  int r, h, row0, rows, a, b, n;
  int cnt[2];  // tiles of each stream
};

template <int NS>
struct Schedule {
  long long g, end;
  int r, qt, h, tile;

  __device__ __forceinline__ bool next(const AttendParams& P, Segment& s) {
    if (g >= end) return false;
    s.q = request_of(P, r);
    while (s.q.rows == 0) s.q = request_of(P, ++r);  // the line ends before the requests do
    s.r = r;
    s.h = h;
    s.row0 = qt * NS * kTile;
    s.rows = min(s.q.rows - s.row0, NS * kTile);
    s.n = tiles_for(P, s.q, s.row0 + s.rows - 1);
    s.a = tile;
    s.b = (int)min((long long)s.n, tile + (end - g));
    if (NS == 1) {
      s.cnt[0] = (s.b - s.a + 1) / 2;
      s.cnt[1] = (s.b - s.a) / 2;
    } else {
      const int n0 = s.rows > kTile ? tiles_for(P, s.q, s.row0 + kTile - 1) : s.n;
      s.cnt[0] = max(0, min(s.b, n0) - s.a);
      s.cnt[1] = s.rows > kTile ? s.b - s.a : 0;
    }
    g += s.b - s.a;
    tile = s.b;
    if (s.b == s.n) {
      tile = 0;
      if (++h == P.c.Hkv) {
        h = 0;
        if ((++qt) * NS * kTile >= s.q.rows) {
          qt = 0;
          ++r;
        }
      }
    }
    return true;
  }
};

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int DP, int NS>
__global__ void __launch_bounds__(kAttThreads, 1)
attend_kernel(const AttendParams P, const __grid_constant__ CUtensorMap k_map,
              const __grid_constant__ CUtensorMap v_map) {
  using L = AttLayout<DP, NS>;
  constexpr int S = L::kStages;
  extern __shared__ unsigned char s_raw[];
  unsigned char* smem = s_raw + ((1024 - (smem_u32(s_raw) & 1023)) & 1023);
  AttMisc& m = *reinterpret_cast<AttMisc*>(smem + L::kMisc);
  float4* scales = reinterpret_cast<float4*>(smem + L::kScales);
  const uint32_t base = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* gave_up = &m.gave_up;

  // ---- setup: barriers, tensor memory, this CTA's share of the line of tiles ----
  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(smem_u32(&m.k_full[i]), 1);
      mbar_init(smem_u32(&m.k_empty[i]), 1);
      mbar_init(smem_u32(&m.v_full[i]), 1);
      mbar_init(smem_u32(&m.v_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&m.s_full[i]), 1);
      mbar_init(smem_u32(&m.p_full[i]), 4);
      mbar_init(smem_u32(&m.o_done[i]), 1);
      mbar_init(smem_u32(&m.q_full[i]), NS == 1 ? 8 : 4);
      mbar_init(smem_u32(&m.q_empty[i]), 1);
    }
    for (int i = 0; i < kScaleSlots; ++i) {
      mbar_init(smem_u32(&m.sc_full[i]), 1);
      mbar_init(smem_u32(&m.sc_empty[i]), NS == 1 ? 4 : 8);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    m.gave_up = 0;
    m.nan_any[0] = m.nan_any[1] = 0;
  }
  if (tid < 256) m.nan_first[tid >> 7][tid & 127] = 0x7fffffff;
  if (warp == 1) tmem_alloc(smem_u32(&m.tmem), 512);
  const int per = (P.B + kAttThreads - 1) / kAttThreads;
  const int r0 = min(P.B, tid * per), r1 = min(P.B, r0 + per);
  long long mine = 0;
  bool bad = false;
  for (int r = r0; r < r1; ++r) {
    const Request q = request_of(P, r);
    for (int row = 0; row < q.rows; row += L::kRows)
      mine += tiles_for(P, q, min(q.rows, row + L::kRows) - 1);
    if (blockIdx.x == 0) bad |= request_bad(P, r);
  }
  if (bad) raise_err(P.err, SD_ERR_KV_RANGE);
  mine *= P.c.Hkv;
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
  for (int w = 0; w < kAttThreads / 32; ++w) {
    if (w < warp) before += m.warp_sum[w];
    total += m.warp_sum[w];
  }
  const long long share = max((long long)P.min_share, (total + gridDim.x - 1) / gridDim.x);
  const long long g0 = min(total, blockIdx.x * share), g1 = min(total, g0 + share);
  if (mine > 0 && before <= g0 && g0 < before + mine) {
    long long at = before;
    for (int r = r0; r < r1; ++r) {
      const Request q = request_of(P, r);
      bool found = false;
      for (int row = 0; row < q.rows; row += L::kRows) {
        const int n = tiles_for(P, q, min(q.rows, row + L::kRows) - 1);
        if (g0 < at + (long long)n * P.c.Hkv) {
          m.start_item[0] = r;
          m.start_item[1] = row / L::kRows;
          m.start_item[2] = (int)(g0 - at);  // head * n + tile
          m.start[0] = n;
          found = true;
          break;
        }
        at += (long long)n * P.c.Hkv;
      }
      if (found) break;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = m.tmem;
  JoinDesc* desc = reinterpret_cast<JoinDesc*>(P.ws) + blockIdx.x;
  float* slots = reinterpret_cast<float*>(P.ws + kMaxCtas * sizeof(JoinDesc));

  Schedule<NS> sched;
  sched.g = g0;
  sched.end = g1;
  sched.r = sched.qt = sched.h = sched.tile = 0;
  if (g0 < g1) {
    const int n = (int)m.start[0];
    sched.r = m.start_item[0];
    sched.qt = m.start_item[1];
    sched.h = m.start_item[2] / n;
    sched.tile = m.start_item[2] % n;
  }
  Segment s;
  const int log2_bs = P.c.log2_bs, bs = 1 << log2_bs;

  if (warp == 0) {
    // ---- loads: lane p of a tile's pages issues that page ----
    const int pages = kTile >> log2_bs;              // of a tile, 1 to 16
    const int batch = 32 / pages < 8 ? 32 / pages : 8;  // tiles whose entries a warp reads at once
    const int my_tile = lane / pages, my_page = lane % pages;
    const uint32_t box = (uint32_t)bs * DP;
    int it = 0;
    bool ok = true;
    while (ok && sched.next(P, s)) {
      const int32_t* table = P.table + (long)s.r * P.max_blocks;
      const int last_page = (s.q.len + bs - 1) >> log2_bs;
      auto entry = [&](int t0) {
        const int pg = ((t0 + my_tile) << (7 - log2_bs)) + my_page;
        int e = -1;
        if (my_tile < batch && t0 + my_tile < s.b && pg < last_page) {
          e = __ldg(table + pg);
          if (e < 0 || e >= P.c.num_blocks) {
            e = -1;
            raise_err(P.err, SD_ERR_KV_RANGE);
          }
        }
        return e < 0 ? P.c.num_blocks : e;  // beyond the tensor: the copy fills in zeros
      };
      int cur = entry(s.a);
      for (int t0 = s.a; ok && t0 < s.b; t0 += batch) {
        const int nxt = t0 + batch < s.b ? entry(t0 + batch) : 0;
        for (int j = 0; j < batch && t0 + j < s.b; ++j, ++it) {
          const int st = it % S;
          const uint32_t par = ((it / S) & 1) ^ 1;
          const uint32_t kf = smem_u32(&m.k_full[st]), vf = smem_u32(&m.v_full[st]);
          ok = mbar_wait_warp(smem_u32(&m.k_empty[st]), par, gave_up);
          if (!ok) break;
          if (lane == 0) mbar_expect_tx(kf, L::kTileBytes);
          __syncwarp();
          if (my_tile == j && my_tile < batch)
            tma_load_4d(base + L::kK + st * L::kTileBytes + my_page * box, &k_map, 0, s.h, 0, cur,
                        kf);
          ok = mbar_wait_warp(smem_u32(&m.v_empty[st]), par, gave_up);
          if (!ok) break;
          if (lane == 0) mbar_expect_tx(vf, L::kTileBytes);
          __syncwarp();
          if (my_tile == j && my_tile < batch)
            tma_load_4d(base + L::kV + st * L::kTileBytes + my_page * box, &v_map, 0, s.h, 0, cur,
                        vf);
        }
        cur = nxt;
      }
    }
  } else if (warp == 1) {
    // ---- products: one thread ----
    if (lane == 0) {
      const uint32_t tS[2] = {tmem, tmem + 128}, tO[2] = {tmem + 256, tmem + 256 + DP};
      constexpr uint32_t qk_desc = mma_desc(kTile, false), pv_desc = mma_desc(DP, true);
      int it = 0, nq[2] = {0, 0}, np[2] = {0, 0};
      bool ok = true;
      auto qk = [&](int st_i, int x, int qi) {  // S[x] = Q[qi] K
        const uint64_t k = smem_desc<DP>(base + L::kK + st_i * L::kTileBytes);
#pragma unroll
        for (int term = 0; term < 2; ++term) {
          const uint64_t a = smem_desc<DP>(base + L::kQ + (qi * 2 + term) * L::kQBytes);
#pragma unroll
          for (int kk = 0; kk < DP / 32; ++kk)
            mma_ss(tS[x], a + kk * 2, k + kk * 2, qk_desc, term + kk > 0);
        }
      };
      auto pv = [&](int st_i, int x, bool add) {  // O[x] += P V
        const uint64_t v = smem_desc<DP>(base + L::kV + st_i * L::kTileBytes);
#pragma unroll
        for (int kk = 0; kk < kTile / 32; ++kk)
#pragma unroll
          for (int term = 0; term < 2; ++term)
            mma_ts(tO[x], tS[x] + kk * 16 + term * 8, v + kk * (32 * DP / 16), pv_desc,
                   add || kk + term > 0);
      };
      while (ok && sched.next(P, s)) {
        const int T = s.b - s.a;
        if (NS == 1) {
          ok = mbar_wait(smem_u32(&m.q_full[0]), nq[0] & 1, gave_up);
          ++nq[0];
          auto do_qk = [&](int j) {
            const int st = (it + j) % S;
            if (!mbar_wait(smem_u32(&m.k_full[st]), ((it + j) / S) & 1, gave_up)) return false;
            tc_fence_after();
            qk(st, j & 1, 0);
            mma_commit(smem_u32(&m.k_empty[st]));
            if (j == T - 1) mma_commit(smem_u32(&m.q_empty[0]));
            mma_commit(smem_u32(&m.s_full[j & 1]));
            return true;
          };
          ok = ok && do_qk(0) && (T < 2 || do_qk(1));
          for (int j = 0; ok && j < T; ++j) {
            const int x = j & 1, st = (it + j) % S;
            ok = mbar_wait(smem_u32(&m.p_full[x]), np[x] & 1, gave_up) &&
                 mbar_wait(smem_u32(&m.v_full[st]), ((it + j) / S) & 1, gave_up);
            if (!ok) break;
            ++np[x];
            tc_fence_after();
            pv(st, x, j >= 2);
            mma_commit(smem_u32(&m.v_empty[st]));
            mma_commit(smem_u32(&m.o_done[x]));
            if (j + 2 < T) ok = do_qk(j + 2);
          }
        } else {
          for (int x = 0; x < 2 && ok; ++x) {
            if (s.cnt[x] > 0) {
              ok = mbar_wait(smem_u32(&m.q_full[x]), nq[x] & 1, gave_up);
              ++nq[x];
            }
          }
          auto do_qk = [&](int j, int x) {
            const int st = (it + j) % S;
            if (!mbar_wait(smem_u32(&m.k_full[st]), ((it + j) / S) & 1, gave_up)) return false;
            tc_fence_after();
            qk(st, x, x);
            if (j == s.cnt[x] - 1) mma_commit(smem_u32(&m.q_empty[x]));
            mma_commit(smem_u32(&m.s_full[x]));
            return true;
          };
          for (int x = 0; x < 2; ++x)
            if (ok && s.cnt[x] > 0) ok = do_qk(0, x);
          if (ok) mma_commit(smem_u32(&m.k_empty[it % S]));
          for (int j = 0; ok && j < T; ++j) {
            const int st = (it + j) % S;
            for (int x = 0; ok && x < 2; ++x) {
              if (j >= s.cnt[x]) continue;
              ok = mbar_wait(smem_u32(&m.p_full[x]), np[x] & 1, gave_up) &&
                   mbar_wait(smem_u32(&m.v_full[st]), ((it + j) / S) & 1, gave_up);
              if (!ok) break;
              ++np[x];
              tc_fence_after();
              pv(st, x, j > 0);
              if (x == 1 || j >= s.cnt[1]) mma_commit(smem_u32(&m.v_empty[st]));
              mma_commit(smem_u32(&m.o_done[x]));
              if (j + 1 < s.cnt[x]) ok = do_qk(j + 1, x);
            }
            if (ok && j + 1 < T) mma_commit(smem_u32(&m.k_empty[(it + j + 1) % S]));
          }
        }
        it += T;
      }
    }
    __syncwarp();
  } else if (warp == 2) {
    // ---- scales: 16 entries a tile, one for 8 tokens; 8 tiles at a time ----
    const int e = lane & 15, half = lane >> 4;
    int it = 0;
    bool ok = true;
    while (ok && sched.next(P, s)) {
      const int32_t* table = P.table + (long)s.r * P.max_blocks;
      for (int t0 = s.a; ok && t0 < s.b; t0 += 8) {
        float ks[4], vs[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const long tok = (long)(t0 + 2 * i + half) * kTile + e * 8;
          ks[i] = 0.f;
          vs[i] = -1.f;  // nothing here
          if (t0 + 2 * i + half < s.b && tok < s.q.len) {
            const int page = __ldg(table + (tok >> log2_bs));
            if (page >= 0 && page < P.c.num_blocks) {
              const long at = (long)page * P.c.Hkv + s.h;
              ks[i] = __ldg(P.c.k_scale + at);
              vs[i] = fmaxf(__ldg(P.c.v_scale + at), 0.f);
              if (vs[i] > 0.f) vs[i] = fmaxf(vs[i], kMinScale);
            }
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            if (t0 + 2 * i + k >= s.b || !ok) break;
            const int slot = it % kScaleSlots;
            ok = mbar_wait_warp(smem_u32(&m.sc_empty[slot]), ((it / kScaleSlots) & 1) ^ 1, gave_up);
            if (!ok) break;
            const uint32_t zero = __ballot_sync(0xffffffffu, half == k && vs[i] == 0.f);
            if (half == k) {
              const bool none = vs[i] < 0.f, z = vs[i] == 0.f;
              scales[slot * 16 + e] =
                  make_float4(ks[i], none ? -INFINITY : z ? kZeroLog2 : log2f(vs[i]),
                              none ? 1.f : z ? kZeroInv : __fdiv_rn(1.f, vs[i]), 0.f);
            }
            if (lane == 0) m.sc_zero[slot] = (int)(k ? zero >> 16 : zero & 0xffffu);
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&m.sc_full[slot]));
            ++it;
          }
        }
      }
    }
  } else if (warp >= 4) {
    // ---- softmax: stream x, one row a thread ----
    const int x = (warp - 4) >> 2, wt = tid - 128 - x * 128;  // thread of its stream
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;        // this warp's quarter of the lanes
    const uint32_t tS = tmem + x * 128 + lanes;
    const uint32_t tO[2] = {tmem + 256 + lanes, tmem + 256 + DP + lanes};
    int it = 0, nq = 0, done[2] = {0, 0}, unit = 0;
    bool ok = true;
    bool continues = false;
    JoinDesc jd;
    jd.pieces = 0;
    // Every thread passes every named barrier, also once a wait has run out (ok is false then, and
    // nothing is computed any more).
    while (sched.next(P, s)) {
      const int T = s.b - s.a;
      const int buf = unit & 1;
      // 1. Q: the rows' two terms into shared memory, their scales
      if (NS == 1 || s.cnt[x] > 0) {
        ok = ok && mbar_wait_warp(smem_u32(&m.q_empty[NS == 1 ? 0 : x]), (nq & 1) ^ 1, gave_up);
        ++nq;
        constexpr int kLanes = DP / 8;  // of a row, 8 values each
        constexpr int kThreads = NS == 1 ? 256 : 128;
        const int t = NS == 1 ? tid - 128 : wt;
        const int c8 = t % kLanes;
        const int qi = NS == 1 ? 0 : x;
        const int rows = ok ? min(kTile, s.rows - qi * kTile) : 0;
        for (int r = t / kLanes; r < ((rows + 31) & ~31); r += kThreads / kLanes) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (r < rows && c8 * 8 < P.c.D) {
            const int row = s.row0 + qi * kTile + r;
            const long tok = s.q.tok0 + row / P.G;
            const int hq = s.h * P.G + row % P.G;
            v = __ldg(reinterpret_cast<const uint4*>(P.q + tok * P.ld_q + hq * P.hs_q + c8 * 8));
          }
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
          float f[8], mag = 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            f[2 * i] = bf16_lo(w[i]);
            f[2 * i + 1] = bf16_hi(w[i]);
            mag = fmaxf(mag, fmaxf(fabsf(f[2 * i]), fabsf(f[2 * i + 1])));
          }
#pragma unroll
          for (int o = kLanes / 2; o > 0; o >>= 1)
            mag = fmaxf(mag, __shfl_xor_sync(0xffffffffu, mag, o));
          // 2^up brings mag to [224, 448]; an infinity stays one and ends as NaN
          const uint32_t mb = __float_as_uint(mag);
          int up = 135 - (int)(mb >> 23) - ((mb & 0x7fffffu) > 0x600000u ? 1 : 0);
          up = mag == 0.f || !(mag < INFINITY) ? 0 : min(up, 120);
          const float mul = __uint_as_float((uint32_t)(up + 127) << 23);
          uint32_t hi[2], lo[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint16_t h2[2], l2[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              float a = f[4 * i + 2 * k] * mul, b = f[4 * i + 2 * k + 1] * mul;
              if (!(fabsf(a) < INFINITY)) a = nanf("");
              if (!(fabsf(b) < INFINITY)) b = nanf("");
              h2[k] = f32_to_e4m3x2(a, b);
              const float2 r2 = e4m3x2_to_f32(h2[k]);
              l2[k] = f32_to_e4m3x2(a - r2.x, b - r2.y);
            }
            hi[i] = h2[0] | (uint32_t)h2[1] << 16;
            lo[i] = l2[0] | (uint32_t)l2[1] << 16;
          }
          // 16-byte chunks of a row are swizzled by the row within its 8-row (or 4-pair) atom
          const int sw = DP == 128 ? r & 7 : (r >> 1) & 3;
          unsigned char* at = smem + L::kQ + qi * 2 * L::kQBytes + r * DP +
                              (((c8 >> 1) ^ sw) << 4) + (c8 & 1) * 8;
          *reinterpret_cast<uint2*>(at) = make_uint2(hi[0], hi[1]);
          *reinterpret_cast<uint2*>(at + L::kQBytes) = make_uint2(lo[0], lo[1]);
          if (c8 == 0)
            m.row_scale[qi * kTile + r] = P.scale * __uint_as_float((uint32_t)(127 - up) << 23);
        }
        fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&m.q_full[NS == 1 ? 0 : x]));
        named_bar(NS == 1 ? 1 : 2 + x, kThreads);  // every row's scale is there
      }
      const int my_rows = NS == 1 ? s.rows : min(kTile, s.rows - x * kTile);  // of this stream
      const int row = s.row0 + (NS == 1 ? 0 : x * kTile) + wt;
      const bool warp_live = (warp & 3) * 32 < my_rows;
      const bool live = wt < my_rows;
      const int lim = seen_by(P, s.q, min(row, s.row0 + s.rows - 1));
      const int min_lim = seen_by(P, s.q, s.row0 + (NS == 1 ? 0 : x * kTile));
      const float rs = m.row_scale[(NS == 1 ? 0 : x * kTile) + wt];
      float M = -INFINITY, Lsum = 0.f;

      // 2. tiles
      for (int j = NS == 1 ? x : 0; ok && j < T; j += NS == 1 ? 2 : 1) {
        const int slot = (it + j) % kScaleSlots;
        ok = mbar_wait_warp(smem_u32(&m.sc_full[slot]), ((it + j) / kScaleSlots) & 1, gave_up);
        if (!ok) break;
        if (NS == 2 && j >= s.cnt[x]) {  // the other stream's alone
          if (lane == 0) mbar_arrive(smem_u32(&m.sc_empty[slot]));
          continue;
        }
        const int t0 = (s.a + j) * kTile;
        const int zero = m.sc_zero[slot];
        const bool masked = t0 + kTile > min_lim;
        if (masked || zero) {
          // V's rows that no row of this call sees become 0, and NaN among the others too (they
          // are noted, for the rows that see them): 0 times NaN is no 0
          const int st = (it + j) % S;
          ok = mbar_wait_warp(smem_u32(&m.v_full[st]), ((it + j) / S) & 1, gave_up);
          if (!ok) break;
          unsigned char* vr = smem + L::kV + st * L::kTileBytes + wt * DP;
          const bool gone = t0 + wt >= s.q.len || ((zero >> (wt >> 3)) & 1);
          const int sw = DP == 128 ? wt & 7 : (wt >> 1) & 3;
#pragma unroll
          for (int ch = 0; ch < DP / 16; ++ch) {
            uint4* p = reinterpret_cast<uint4*>(vr + ((ch ^ sw) << 4));
            if (gone) {
              *p = make_uint4(0, 0, 0, 0);
              continue;
            }
            const uint4 q = *p;
            uint32_t w[4] = {q.x, q.y, q.z, q.w};
            uint32_t any = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              any |= ((w[i] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
            if (any && masked) {
              for (int b = 0; b < 16; ++b)
                if (((w[b >> 2] >> ((b & 3) * 8)) & 0x7f) == 0x7f) {
                  atomicMin(&m.nan_first[buf][ch * 16 + b], t0 + wt);
                  w[b >> 2] &= ~(0xffu << ((b & 3) * 8));
                }
              m.nan_any[buf] = 1;
              __threadfence_block();
              *p = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
          fence_async_shared();
        }
        ok = mbar_wait_warp(smem_u32(&m.s_full[x]), done[x] & 1, gave_up);
        if (!ok) break;
        tc_fence_after();
        if (warp_live) {
          const float4* sc = scales + slot * 16;
          const int edge = lim - t0;  // columns from here on are masked
          float mx = -INFINITY;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t v[32];
            tmem_ld32(tS + c * 32, v);
            tmem_wait_ld();
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              const float4 f = sc[c * 4 + g];
              float b = -INFINITY;
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float a = __uint_as_float(v[g * 8 + i]);
                b = fmaxf(b, masked && c * 32 + g * 8 + i >= edge ? -INFINITY : a);
              }
              // a column group without a token: 0 times its zeros, and -inf
              const float y = fmaf(b, f.x * rs, f.y);
              mx = fmaxf(mx, y);
            }
          }
          // P stays within e4m3 while M is at most 0.75 behind
          const bool grow = mx > M + 0.75f;
          if (__any_sync(0xffffffffu, grow)) {
            const float Mn = fmaxf(M, mx);
            if (done[x] > 0 && j >= (NS == 1 ? 2 : 1)) {
              const float fac = M == -INFINITY ? 0.f : ex2f(M - Mn);
              ok = mbar_wait_warp(smem_u32(&m.o_done[x]), (done[x] - 1) & 1, gave_up);
              if (!ok) break;
              tc_fence_after();
#pragma unroll
              for (int c = 0; c < DP / 32; ++c) {
                uint32_t v[32];
                tmem_ld32(tO[x] + c * 32, v);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  v[i] = __float_as_uint(__uint_as_float(v[i]) * fac);
                tmem_st32(tO[x] + c * 32, v);
              }
              Lsum *= fac;
            }
            M = Mn;
          }
          const float shift = 8.f - (M == -INFINITY ? 0.f : M);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t v[32], o[16];
            tmem_ld32(tS + c * 32, v);
            tmem_wait_ld();
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              const float4 f = sc[c * 4 + g];
              const float k = f.x * rs, add = f.y + shift;
              float sum = 0.f;
              uint16_t p1[4], p2[4];
#pragma unroll
              for (int i = 0; i < 8; i += 2) {
                float p[2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                  const float a = __uint_as_float(v[g * 8 + i + u]);
                  p[u] = ex2f(fmaf(a, k, add));
                  if (masked && c * 32 + g * 8 + i + u >= edge) p[u] = 0.f;
                  sum += p[u];
                }
                // the leading 4 significant bits, and the rest
                const float a1 = __uint_as_float(__float_as_uint(p[0]) & 0xfff00000u);
                const float b1 = __uint_as_float(__float_as_uint(p[1]) & 0xfff00000u);
                p1[i >> 1] = f32_to_e4m3x2(a1, b1);
                p2[i >> 1] = f32_to_e4m3x2(p[0] - a1, p[1] - b1);
              }
              Lsum = fmaf(sum, f.z, Lsum);
              o[g * 2] = p1[0] | (uint32_t)p1[1] << 16;
              o[g * 2 + 1] = p1[2] | (uint32_t)p1[3] << 16;
              o[8 + g * 2] = p2[0] | (uint32_t)p2[1] << 16;
              o[8 + g * 2 + 1] = p2[2] | (uint32_t)p2[3] << 16;
            }
            tmem_st16(tS + c * 16, o);
          }
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&m.sc_empty[slot]));
          mbar_arrive(smem_u32(&m.p_full[x]));
        }
        ++done[x];
      }
      if (NS == 1) done[x ^ 1] += s.cnt[x ^ 1];

      // 3. the unit's (or this part's) result
      const bool split = s.a > 0 || s.b < s.n;
      const int cnt_b = NS == 1 ? s.cnt[1] : 0;
      if (NS == 1) {
        ok = ok && mbar_wait_warp(smem_u32(&m.o_done[0]), (done[0] - 1) & 1, gave_up);
        if (cnt_b > 0)
          ok = ok && mbar_wait_warp(smem_u32(&m.o_done[1]), (done[1] - 1) & 1, gave_up);
        m.ml[x][wt] = make_float2(M, Lsum);
      } else if (s.cnt[x] > 0) {
        ok = ok && mbar_wait_warp(smem_u32(&m.o_done[x]), (done[x] - 1) & 1, gave_up);
      }
      tc_fence_after();
      named_bar(1, 256);
      const bool has_nan = m.nan_any[buf] != 0;
      if (tid - 128 < 128) m.nan_first[buf ^ 1][tid - 128] = 0x7fffffff;
      if (tid == 128) m.nan_any[buf ^ 1] = 0;
      float wa = 1.f, wb = 0.f, Mt = M, Lt = Lsum;
      if (NS == 1) {
        const float2 a = m.ml[0][wt], b = m.ml[1][wt];
        if (cnt_b > 0) {
          Mt = fmaxf(a.x, b.x);
          wa = a.x == Mt ? 1.f : ex2f(a.x - Mt);
          wb = b.x == Mt ? 1.f : ex2f(b.x - Mt);
          Lt = a.y * wa + b.y * wb;
        } else {
          Mt = a.x;
          Lt = a.y;
        }
      }
      const float inv = Lt == 0.f ? 0.f : 1.f / Lt;
      const float lse2 = Lt == 0.f ? -INFINITY : Mt - 8.f + log2f(Lt);
      wa *= inv;
      wb *= inv;
      const int unit_row = (NS == 1 ? 0 : x * kTile) + wt;
      const long tok = s.q.tok0 + row / P.G;
      const int hq = s.h * P.G + row % P.G;
      float* slot = slots + (2L * blockIdx.x + (s.a > 0 ? 0 : 1)) * L::kSlotFloats;
      const bool mine_any = NS == 1 || s.cnt[x] > 0;
      if (ok && warp_live && my_rows > 0) {
        constexpr int kCols = NS == 1 ? DP / 2 : DP;  // this thread's share of the row
        const int c0 = NS == 1 ? x * kCols : 0;
        if (mine_any) {
#pragma unroll
          for (int c = 0; c < kCols; c += 32) {
            uint32_t u[32], w[32];
            tmem_ld32(tO[NS == 1 ? 0 : x] + c0 + c, u);
            if (NS == 1 && cnt_b > 0) tmem_ld32(tO[1] + c0 + c, w);
            tmem_wait_ld();
            if (!live) continue;
            float o[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              o[i] = __uint_as_float(u[i]) * wa;
              if (NS == 1 && cnt_b > 0) o[i] = fmaf(__uint_as_float(w[i]), wb, o[i]);
            }
            if (has_nan) {
              for (int i = 0; i < 32; ++i)
                if (m.nan_first[buf][c0 + c + i] < lim) o[i] = nanf("");
            }
            if (split) {
              float4* p = reinterpret_cast<float4*>(slot + (long)unit_row * DP + c0 + c);
#pragma unroll
              for (int i = 0; i < 8; ++i)
                p[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
            } else {
              uint16_t* p = P.out + tok * P.ld_out + hq * P.hs_out + c0 + c;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if (c0 + c + i * 8 < P.c.D) {
                  uint32_t b[4];
#pragma unroll
                  for (int k = 0; k < 4; ++k) {
                    const __nv_bfloat162 h2 =
                        __floats2bfloat162_rn(o[i * 8 + 2 * k], o[i * 8 + 2 * k + 1]);
                    b[k] = *reinterpret_cast<const uint32_t*>(&h2);
                  }
                  *reinterpret_cast<uint4*>(p + i * 8) = make_uint4(b[0], b[1], b[2], b[3]);
                }
              }
            }
          }
        }
        if (live && (NS == 2 || x == 0)) {
          if (split) slot[(long)L::kRows * DP + unit_row] = mine_any ? lse2 : -INFINITY;
          else if (P.lse) P.lse[tok * P.Hq + hq] = lse2 * kLn2F;
        }
      }
      if (s.a == 0 && s.b < s.n) {  // begun here, ended by a later CTA
        continues = true;
        const long long first = sched.g - (s.b - s.a);  // the unit's place on the line
        jd.pieces = (int)((first + s.n - 1) / share - blockIdx.x + 1);
        jd.tok0 = s.q.tok0;
        jd.head = s.h;
        jd.row0 = s.row0;
        jd.rows = s.rows;
      }
      tc_fence_before();
      named_bar(1, 256);  // both streams have read the accumulators
      it += T;
      ++unit;
    }
    if (tid == 128) {
      if (!continues) jd.pieces = 0;
      *desc = jd;
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (m.gave_up) {
    // a wait ran out: the copies in flight get some milliseconds before the memory is given up
    if (tid == 0) raise_err(P.err, SD_ERR_WAIT);
    const long long t = clock64();
    while (clock64() - t < 20000000LL) __nanosleep(1000);
    __syncthreads();
  }
  tc_fence_after();
  if (warp == 1) tmem_free(tmem, 512);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Joins the parts of a unit that several CTAs shared: one warp a row, parts in their order.
template <int DP, int NS>
__global__ void __launch_bounds__(256) attend_join_kernel(const AttendParams P) {
  using L = AttLayout<DP, NS>;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const JoinDesc d = reinterpret_cast<const JoinDesc*>(P.ws)[blockIdx.x];
  const int r = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (d.pieces == 0 || r >= d.rows) return;
  const float* slots = reinterpret_cast<const float*>(P.ws + kMaxCtas * sizeof(JoinDesc));
  auto slot = [&](int p) {
    return slots + (2L * (blockIdx.x + p) + (p == 0 ? 1 : 0)) * L::kSlotFloats;
  };
  float mx = -INFINITY;
  for (int p = lane; p < d.pieces; p += 32)
    mx = fmaxf(mx, __ldcg(slot(p) + (long)L::kRows * DP + r));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  constexpr int V = DP / 32;
  float acc[V], sum = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.f;
#pragma unroll 4
  for (int p = 0; p < d.pieces; ++p) {
    const float* s = slot(p);
    const float l = __ldcg(s + (long)L::kRows * DP + r);
    float v[V];
    if (V == 4) {
      const float4 f = __ldcg(reinterpret_cast<const float4*>(s + (long)r * DP) + lane);
      v[0] = f.x;
      v[1] = f.y;
      v[V > 2 ? 2 : 0] = f.z;
      v[V > 2 ? 3 : 0] = f.w;
    } else {
      const float2 f = __ldcg(reinterpret_cast<const float2*>(s + (long)r * DP) + lane);
      v[0] = f.x;
      v[1] = f.y;
    }
    if (l == -INFINITY) continue;  // nothing seen (and nothing written) in this part
    const float w = l == mx ? 1.f : ex2f(l - mx);
    sum += w;
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = fmaf(w, v[i], acc[i]);
  }
  const int row = d.row0 + r;
  const long tok = d.tok0 + row / P.G;
  const int hq = d.head * P.G + row % P.G;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  uint16_t* out = P.out + tok * P.ld_out + hq * P.hs_out + lane * V;
  if (lane * V < P.c.D) {
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const __nv_bfloat162 h2 = __floats2bfloat162_rn(acc[i] * inv, acc[i + 1] * inv);
      *reinterpret_cast<uint32_t*>(out + i) = *reinterpret_cast<const uint32_t*>(&h2);
    }
  }
  if (P.lse && lane == 0)
    P.lse[tok * P.Hq + hq] = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * kLn2F;
}

// ---------------------------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------------------------
typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeTiled encode_tiled() {
  static EncodeTiled fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return (EncodeTiled)p;
  }();
  return fn;
}

// [page][slot][head][d] bytes; a box is one page (or a tile of it) of one head, D filled up with
// zeros to DP.
static bool cache_map(CUtensorMap* map, const void* p, const KvCache& c, int DP) {
  const int bs = 1 << c.log2_bs;
  const cuuint64_t dims[4] = {(cuuint64_t)c.D, (cuuint64_t)c.Hkv, (cuuint64_t)bs,
                              (cuuint64_t)c.num_blocks};
  const cuuint64_t strides[3] = {(cuuint64_t)c.st_head, (cuuint64_t)c.st_tok,
                                 (cuuint64_t)c.st_block};
  const cuuint32_t box[4] = {(cuuint32_t)DP, 1, (cuuint32_t)bs, 1};
  const cuuint32_t one[4] = {1, 1, 1, 1};
  const EncodeTiled fn = encode_tiled();
  return fn && fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(p), dims, strides, box,
                  one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  DP == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

static int sm_count() {
  static int count[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  if (count[dev] == 0) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    count[dev] = n;
  }
  return count[dev];
}

template <int DP, int NS>
static int launch_attend(const AttendParams& P, const CUtensorMap& km, const CUtensorMap& vm,
                         int ctas, bool join, cudaStream_t stream) {
  using L = AttLayout<DP, NS>;
  constexpr int smem = L::kMisc + (int)sizeof(AttMisc) + 1024;
  static_assert(smem <= 227 * 1024, "shared memory of one CTA");
  static bool set[64];  // per device
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return SD_E_DEVICE;
  if (!set[dev]) {
    if (cudaFuncSetAttribute(attend_kernel<DP, NS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             smem) != cudaSuccess)
      return SD_E_LAUNCH;
    set[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas, 1, 1);
  cfg.blockDim = dim3(kAttThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  if (cudaLaunchKernelEx(&cfg, attend_kernel<DP, NS>, P, km, vm) != cudaSuccess)
    return SD_E_LAUNCH;
  if (!join) return SD_OK;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t jc = {};
  jc.gridDim = dim3((unsigned)ctas, (unsigned)(L::kRows / 8), 1);
  jc.blockDim = dim3(256, 1, 1);
  jc.stream = stream;
  jc.attrs = attr;
  jc.numAttrs = 1;
  return cudaLaunchKernelEx(&jc, attend_join_kernel<DP, NS>, P) == cudaSuccess ? SD_OK
                                                                               : SD_E_LAUNCH;
}

}  // namespace sdk

extern "C" size_t sd_kv_attend_workspace_launch(int D) {
  const long slot = D <= 64 ? sdk::AttLayout<64, 2>::kSlotFloats : sdk::AttLayout<128, 2>::kSlotFloats;
  return sdk::kMaxCtas * sizeof(sdk::JoinDesc) + (size_t)2 * sdk::kMaxCtas * slot * sizeof(float);
}

extern "C" int sd_kv_attend_launch(int B, int n, int max_q, int Hq, int Hkv, int D, const void* q,
                                   long ld_q, long hs_q, const void* k_cache, const void* v_cache,
                                   long st_block, long st_tok, long st_head, const float* k_scale,
                                   const float* v_scale, int num_blocks, int log2_bs,
                                   const int32_t* table, int max_blocks, const int32_t* ctx,
                                   const int32_t* cu, float sm_scale, int causal, void* out,
                                   long ld_out, long hs_out, float* lse, void* workspace,
                                   int32_t* err, cudaStream_t stream) {
  sdk::AttendParams P;
  P.c = sdk::KvCache{(const uint8_t*)k_cache, (const uint8_t*)v_cache, k_scale, v_scale,
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
  P.table = table;
  P.ctx = ctx;
  P.cu = cu;
  P.scale = sm_scale * sdk::kLog2eF;
  P.out = (uint16_t*)out;
  P.ld_out = ld_out;
  P.hs_out = hs_out;
  P.lse = lse;
  P.ws = (unsigned char*)workspace;
  P.err = err;
  P.min_share = 4;
  const int sms = sdk::sm_count();
  if (sms < 1) return SD_E_DEVICE;
  const int ctas = sms < sdk::kMaxCtas ? sms : sdk::kMaxCtas;
  CUtensorMap km, vm;
  const int DP = D <= 64 ? 64 : 128;
  if (!sdk::cache_map(&km, k_cache, P.c, DP) || !sdk::cache_map(&vm, v_cache, P.c, DP))
    return SD_E_SHAPE;
  // units of one tile are never shared
  const bool join = ((long)max_blocks << log2_bs) > sdk::kTile;
  const bool many = (long)max_q * P.G > sdk::kTile;
  if (DP == 64)
    return many ? sdk::launch_attend<64, 2>(P, km, vm, ctas, join, stream)
                : sdk::launch_attend<64, 1>(P, km, vm, ctas, join, stream);
  return many ? sdk::launch_attend<128, 2>(P, km, vm, ctas, join, stream)
              : sdk::launch_attend<128, 1>(P, km, vm, ctas, join, stream);
}
