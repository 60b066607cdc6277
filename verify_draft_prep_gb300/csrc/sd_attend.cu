// sd_attend.cu -- attention over the paged 8-bit cache (sd_kv_attend), on the fifth-generation
// tensor cores.
//
// Query token i of request r stands at position ctx_lens[r] - n_q + i and sees every token up to
// its own position (causal) or all of them. With S = sm_scale q k, M the running maximum and L
// the running sum of the exponentials: O = sum e^(S - M) v / L, lse = M + ln L.
//
// The cache's bytes go to the tensor cores as they are, without being converted: an e4m3 value has
// 4 significant bits and bf16 has 8, so q is split into two e4m3 terms, q = q1 + q2 (after a power
// of two per row brings its largest magnitude to [224, 448]; exact but for what lies below 2^-17 of
// that), and each weight into an e5m2 and an e4m3 term, P = P1 + P2. Two 8-bit products take the
// time of one bf16 product, and K and V cost half the shared memory and no instructions. A page's
// scales enter as numbers per 8 columns of S: with y = log2(e) S + log2(v_scale),
//   P = 2^(y - M + kShift),  O = sum P v_byte,  L = sum P / v_scale,
// M a reference that keeps near the tiles' largest y, so that one exponential serves both sums.
//
// A unit is one request's 128 (or 256) rows of one KV head; a row is a query token and one of the
// Hq / Hkv heads that share the KV head. All units' tiles of 128 tokens form one line, which the
// CTAs (one per SM) divide evenly, whatever the lengths of the requests: a unit that several CTAs
// share leaves its parts in the workspace and attend_join_kernel joins them in a fixed order.
// Within a CTA: warps 0 and 2 load pages (TMA), warp 1 issues the products, warp 3 fetches the
// scales and the next unit's queries, two groups of four warps turn S into P, one row a thread. The
// groups are two streams that keep the tensor cores busy in turn: with few rows they take alternate
// tiles of the same rows (and the accumulators are joined at the unit's end), with many they take
// 128 rows each of the same tiles, which halves the traffic of K and V.
//
// What bounds it (measured, 8 heads of K and V, pages of 16):
//   - 256 requests of 8 slots, 32 heads of 128, 1000 to 16000 tokens: 890 us in short runs, 76% of
//     the copy rate, and 960 to 1020 once the power limit lowers the clocks after some tenths of a
//     second.
//   - 64 requests of 6 slots, 64 heads of 64, 512 to 8192 tokens: 120 us against 40 of memory, 128
//     drafter requests of 8 to 16 slots 411 us against 109, a prompt of 8192 tokens of 32 heads of 128
//     640 us against 278 of products. No unit is half busy (64 requests: issue slots 42%, memory 28%,
//     tensor cores 25%; prompt: 48%, 3%, 38%). What takes the time is a stream's chain S -> P -> PV ->
//     next S: P takes the place of the only S, and only two streams cover for each other. A unit's
//     own cost (kUnitCost) is a sixth of the line of 64 requests.
//   - One token at 32000, 32 heads of 128: 31 us in a graph against 9.7 of memory: 14 tiles a CTA do
//     not hide the setup, the first pages' latency and the join of 19 parts.
// Softmax beside a product that takes both operands from shared memory is 2.3 times slower; that is
// why heads of 64 keep Q in tensor memory.

#include <atomic>

#include "sd_kv.cuh"
#include "sd_tc.cuh"

namespace sdk {

constexpr int kTile = 128;                 // tokens of a tile, rows of a stream
constexpr int kAttThreads = 384;
constexpr int kMaxCtas = 160;
constexpr int kScaleSlots = 16;            // tiles of scales in flight
// A page whose V scale is 0 holds zeros: its tokens weigh in L only. They are given a scale far below
// that of pages with values of any ordinary size, so that those keep P's full precision.
constexpr float kZeroLog2 = -60.f, kZeroInv = 1152921504606846976.f;
// P = 2^(y - M + kShift), M the row's reference, as P1 + P2: P1 is P to 3 significant bits (e5m2),
// P2 the rest, at most 2^-3 of P's binade, to 4 (e4m3). Below 2^12 P2 stays within e4m3's 448. P has 8
// significant bits down to 2^-2, where P2 reaches e4m3's finest step of 2^-9, and fewer below, 3 down
// to 2^-14. A long context can hold thousands of weights far below one dominant token's, which
// together are the answer where that token's V is small. So M follows the tiles both ways: up where a
// tile's largest y passes M + kSlack, down where it lies below M - kFall, and every tile's largest P is
// between 2^(kShift - kFall) = 2^-2 and 2^(kShift + kSlack) < 2^12. The smaller kFall, the more bits the
// small weights keep and the more often the accumulator is rescaled: with 9, 12, 14 and no fall 64
// requests take 124, 122, 122, 120 us, 256 requests 896, 889, 884, 871, drafter batch 418, 413, 410,
// 404, prompt 648, 640, 633, 608; at 12 the largest weight of every tile has all of its 8 bits. M
// falls to kAbove above the tile's largest y, so that the next tiles find room on either side, and
// kDeepest at most below the largest M so far, so that the accumulator (up to 2^21 a token at the
// largest M) stays within fp32; nor beyond kMaxL for L, which a small V scale enlarges.
constexpr float kShift = 10.f, kSlack = 1.9f, kFall = 12.f, kAbove = 2.f, kDeepest = 60.f;
constexpr float kMaxL = 1e30f;
constexpr float kTiny = 1.17549435e-38f;  // -inf times it is -inf, S times it is nothing
constexpr float kLog2eF = 1.4426950408889634f, kLn2F = 0.6931471805599453f;

struct AttendParams {
  KvCache c;
  int B, n, Hq, G, max_blocks, causal, min_share, out_32;  // out_32: every 16 values of out 32-byte aligned
  unsigned long long g_magic;  // ceil(2^64 / G); 0 for G = 1
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

// R: how often a unit's rows stand in the 128 lanes (each copy takes 1/R of a tile's columns).
// NS: Q tiles of a unit (1: both streams share it, 2: one each).
template <int DP, int NS, int R>
struct AttLayout {
  static constexpr int kRows = NS * kTile / R;      // of a unit
  // Tensor memory, 512 columns: S of both streams (P takes its place), O of both, and with heads of
  // 64 also Q, a copy for each stream: a product that takes Q from there reads half as much shared
  // memory, which the softmax, the barriers and the loads need, too.
  static constexpr bool kQTm = DP == 64;
  static constexpr int kTmO = 256, kTmQ = 256 + 2 * DP;
  static constexpr int kQBytes = kTile * DP;        // one term of one Q tile
  static constexpr int kTileBytes = kTile * DP;     // K or V of one tile
  // Tiles in flight, as many as fit. V's stay longer (until P is formed and used) than K's.
  static constexpr int kKStages = DP == 64 ? 8 : (NS == 1 ? 3 : 4);
  static constexpr int kVStages = DP == 64 ? 12 : (NS == 1 ? 5 : 4);
  static constexpr int kQ = 0;                      // two buffers (NS = 1), or two tiles
  static constexpr int kK = kQ + (kQTm ? 0 : 2 * 2 * kQBytes);
  static constexpr int kV = kK + kKStages * kTileBytes;
  static constexpr int kScales = kV + kVStages * kTileBytes;
  static constexpr int kJoinCols = DP == 64 ? 32 : 16;           // joined at a time
  static constexpr int kJoin = kScales + kScaleSlots * 16 * 16;  // [8 warps][32 rows][those + 1]
  static constexpr int kMisc = kJoin + (R > 1 ? 8 * 32 * (kJoinCols + 1) * 4 : 0);
  static constexpr long kSlotFloats = (long)kRows * DP + kRows;
};

struct AttMisc {
  uint64_t k_full[12], k_empty[12], v_full[12], v_empty[12];
  uint64_t s_full[2], p_full[2], o_done[2], q_full[2], q_empty[2];
  uint64_t sc_full[kScaleSlots], sc_empty[kScaleSlots];
  uint32_t sc_zero[kScaleSlots];  // bit e: entry e's V scale is zero, bit 16 + e: its K scale
  float row_scale[2 * kTile];
  float2 ml[2][kTile];        // (M, L) of both streams; before a unit's end (the largest M so far, -)
  int nan_first[2][128];      // first token with a NaN in dimension d of V, of a masked tile
  int nan_any[2];
  int start_item[4];          // of the schedule
  long long g0, share;
  long long warp_sum[kAttThreads / 32];
  uint32_t tmem;
  int gave_up;
};

// row / G and row % G, exactly for every 32-bit row.
__device__ __forceinline__ int2 token_head(const AttendParams& P, int row) {
  const int t = P.g_magic ? (int)__umul64hi((unsigned long long)row, P.g_magic) : row;
  return make_int2(t, row - t * P.G);
}

struct Request {
  int tok0, n_q, rows, len, off;
};

// Tokens that a request's table covers; positions of a tile's end stay within int.
__device__ __forceinline__ long covered(const AttendParams& P) {
  return min((long)P.max_blocks << P.c.log2_bs, 2147483648L - 2 * kTile);
}

__device__ __forceinline__ Request request_of(const AttendParams& P, int r) {
  Request q;
  // (plain loads: a read-only one may be moved up before the wait for the work before this kernel)
  const int a = P.cu[r], b = P.cu[r + 1];
  const int lo = min(max(a, 0), P.n), hi = min(max(b, lo), P.n);
  q.tok0 = lo;
  q.n_q = hi - lo;
  q.rows = q.n_q * P.G;
  const int ctx = P.ctx[r];
  q.len = ctx < 0 ? 0 : (int)min((long)ctx, covered(P));
  q.off = (int)max((long)ctx - q.n_q, -2147483647L);
  return q;
}

__device__ __forceinline__ bool request_bad(const AttendParams& P, int r) {
  const int a = P.cu[r], b = P.cu[r + 1], ctx = P.ctx[r];
  return a < 0 || b < a || b > P.n || ctx < 0 || ctx > covered(P);
}

// Tokens that a row sees.
__device__ __forceinline__ int seen_by(const AttendParams& P, const Request& q, int row) {
  if (!P.causal) return q.len;
  const long t = (long)q.off + token_head(P, row).x + 1;
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
  int cnt0, cnt1;   // tiles of each stream
  long long first;  // the unit's first tile on the line
};

// Every unit takes kUnitCost places on the line before its tiles, for what it costs beside them (its
// queries, its result), so that CTAs with many short units get fewer tiles. With 2, 4, 6, 8 and 16:
// 64 requests 127, 124, 122, 123, 131 us; 256 requests 897, 890, 890, 890, 894; drafter batch 417, 407,
// 413, 423, 474; prompt 883, 640, 640, 651, 697; one token 34 everywhere but 36 with 16.
constexpr int kUnitCost = 6;

// The order of the line: heads outermost (requests, then their Q tiles inside), or, with two Q tiles,
// innermost. Outermost against innermost: 64 requests 122 to 125 us, drafter batch 413 to 425, 256
// requests 890 to 888, prompt (two Q tiles) 643 to 640.
template <int NS>
constexpr bool kHeadsInside = NS == 2;

template <int NS, int ROWS>
struct Schedule {
  long long g, end;  // this CTA's part of the line
  int r, qt, h, off; // the unit at g, and how far into its places g lies

  __device__ __forceinline__ bool next(const AttendParams& P, Segment& s) {
    while (g < end) {
      if (!kHeadsInside<NS> && r == P.B) {
        r = 0;
        ++h;
      }
      s.q = request_of(P, r);
      if (s.q.rows == 0) {
        ++r;
        continue;
      }
      s.r = r;
      s.h = h;
      s.row0 = qt * ROWS;
      s.rows = min(s.q.rows - s.row0, ROWS);
      s.n = tiles_for(P, s.q, s.row0 + s.rows - 1);
      s.first = g - off + kUnitCost;
      const int take = (int)min((long long)(s.n + kUnitCost - off), end - g);
      s.a = max(0, off - kUnitCost);
      s.b = max(0, off + take - kUnitCost);
      g += take;
      off += take;
      if (off == s.n + kUnitCost) {
        off = 0;
        if (!kHeadsInside<NS> || ++h == P.c.Hkv) {
          if (kHeadsInside<NS>) h = 0;
          if ((++qt) * ROWS >= s.q.rows) {
            qt = 0;
            ++r;
          }
        }
      }
      if (s.b <= s.a) continue;
      if (NS == 1) {
        s.cnt0 = (s.b - s.a + 1) / 2;
        s.cnt1 = (s.b - s.a) / 2;
      } else {
        const int n0 = s.rows > kTile ? tiles_for(P, s.q, s.row0 + kTile - 1) : s.n;
        s.cnt0 = max(0, min(s.b, n0) - s.a);
        s.cnt1 = s.rows > kTile ? s.b - s.a : 0;
      }
      return true;
    }
    return false;
  }
};

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 2^up that brings a row's largest magnitude (a bf16 pattern) to [224, 448]; a row with an infinity
// or a NaN becomes NaN, as its softmax is.
__device__ __forceinline__ float q_factor(uint32_t mg, int& up) {
  up = 135 - (int)(mg >> 7) - ((mg & 0x7fu) > 0x60u ? 1 : 0);
  up = mg == 0 ? 0 : min(up, 64);
  return mg >= 0x7f80u ? nanf("") : __uint_as_float((uint32_t)(up + 127) << 23);
}

// What brings a row's scores back to sm_scale q . k, in binades; NaN for a row of NaN.
__device__ __forceinline__ float row_scale_of(const AttendParams& P, float mul, int up) {
  return mul != mul ? mul : P.scale * __uint_as_float((uint32_t)(127 - up) << 23);
}

// 8 bf16 times mul as two e4m3 terms: the leading 4 significant bits, and the rest.
__device__ __forceinline__ void split8(const uint4& v, float mul, uint32_t* hi, uint32_t* lo) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float f[4], h[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      f[u] = (u & 1 ? bf16_hi(w[2 * k + (u >> 1)]) : bf16_lo(w[2 * k + (u >> 1)])) * mul;
      h[u] = __uint_as_float(__float_as_uint(f[u]) & 0xfff00000u);
    }
    hi[k] = f32_to_e4m3x4(h[0], h[1], h[2], h[3]);
    lo[k] = f32_to_e4m3x4(f[0] - h[0], f[1] - h[1], f[2] - h[2], f[3] - h[3]);
  }
}

// Q rows [first, first + count) of a unit, one 8-value part a thread, as two e4m3 terms into the
// swizzled operand at q (and q + kQBytes), R copies of them, with the rows' scales. `rows` valid.
template <int DP, int R, int THREADS>
__device__ __forceinline__ void load_q(const AttendParams& P, const Segment& s, int row0, int rows,
                                       unsigned char* q, float* row_scale, int t) {
  constexpr int kLanes = DP / 8, kPerPass = THREADS / kLanes;
  constexpr int kAhead = 4;  // loads in flight, while the code of one row stays small
  const int c8 = t % kLanes;
  const int padded = (rows + 31) & ~31;
  auto fetch = [&](int r) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (r < rows && c8 * 8 < P.c.D) {
      const int row = row0 + r;
      const int2 th = token_head(P, row);
      const long tok = s.q.tok0 + th.x;
      const int hq = s.h * P.G + th.y;
      v = __ldg(reinterpret_cast<const uint4*>(P.q + tok * P.ld_q + hq * P.hs_q + c8 * 8));
    }
    return v;
  };
  uint4 q4[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) q4[i] = fetch(i * kPerPass + t / kLanes);
#pragma unroll 2
  for (int rb = 0; rb < padded; rb += kPerPass) {
    const int r = rb + t / kLanes;
    const uint4 v = q4[0];
#pragma unroll
    for (int i = 0; i + 1 < kAhead; ++i) q4[i] = q4[i + 1];
    q4[kAhead - 1] = fetch(r + kAhead * kPerPass);
    {
      uint32_t mg = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                             __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
      mg = max(mg & 0xffffu, mg >> 16);
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) mg = max(mg, __shfl_xor_sync(0xffffffffu, mg, o));
      int up;
      const float mul = q_factor(mg, up);
      uint32_t hi[2], lo[2];
      split8(v, mul, hi, lo);
      // 16-byte chunks of a row are swizzled by the row within its 8-row (or 4-pair) atom; the
      // copies lie whole atoms apart
      const int sw = DP == 128 ? r & 7 : (r >> 1) & 3;
      unsigned char* at = q + r * DP + (((c8 >> 1) ^ sw) << 4) + (c8 & 1) * 8;
#pragma unroll
      for (int k = 0; k < R; ++k) {
        *reinterpret_cast<uint2*>(at + k * (kTile / R) * DP) = make_uint2(hi[0], hi[1]);
        *reinterpret_cast<uint2*>(at + k * (kTile / R) * DP + kTile * DP) =
            make_uint2(lo[0], lo[1]);
      }
      if (c8 == 0) row_scale[r] = row_scale_of(P, mul, up);
    }
  }
}

// One row of Q (up to 64 values), by the thread of its lane, as two e4m3 terms into tensor memory:
// 16 columns each, 4 values a column. Returns the row's scale.
__device__ __forceinline__ float q_to_tmem(const AttendParams& P, const Segment& s, int row,
                                           bool live, uint32_t dst) {
  uint4 v[8];
  const int2 th = token_head(P, row);
  const uint16_t* q = P.q + (long)(s.q.tok0 + th.x) * P.ld_q + (long)(s.h * P.G + th.y) * P.hs_q;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    v[i] = live && i * 8 < P.c.D ? __ldg(reinterpret_cast<const uint4*>(q) + i)
                                 : make_uint4(0, 0, 0, 0);
  uint32_t mg = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    mg = __vmaxu2(mg, __vmaxu2(__vmaxu2(v[i].x & 0x7fff7fffu, v[i].y & 0x7fff7fffu),
                               __vmaxu2(v[i].z & 0x7fff7fffu, v[i].w & 0x7fff7fffu)));
  mg = max(mg & 0xffffu, mg >> 16);
  int up;
  const float mul = q_factor(mg, up);
  __syncwarp();  // (the lanes without a row have read nothing)
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t o[16];  // 8 words of the first term, 8 of the second
#pragma unroll
    for (int i = 0; i < 4; ++i) split8(v[half * 4 + i], mul, o + 2 * i, o + 8 + 2 * i);
    tmem_st8(dst + half * 8, o);
    tmem_st8(dst + 16 + half * 8, o + 8);
  }
  tmem_wait_st();
  return row_scale_of(P, mul, up);
}

// One row of Q (up to 128 values) by a thread of its own, into the swizzled operand in shared memory
// (lane: the row there). Returns the row's scale.
__device__ __forceinline__ float q_to_smem(const AttendParams& P, const Segment& s, int row,
                                           bool live, int lane, unsigned char* q_smem) {
  uint4 v[16];
  const int2 th = token_head(P, row);
  const uint16_t* q = P.q + (long)(s.q.tok0 + th.x) * P.ld_q + (long)(s.h * P.G + th.y) * P.hs_q;
#pragma unroll
  for (int i = 0; i < 16; ++i)
    v[i] = live && i * 8 < P.c.D ? __ldg(reinterpret_cast<const uint4*>(q) + i)
                                 : make_uint4(0, 0, 0, 0);
  uint32_t mg = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i)
    mg = __vmaxu2(mg, __vmaxu2(__vmaxu2(v[i].x & 0x7fff7fffu, v[i].y & 0x7fff7fffu),
                               __vmaxu2(v[i].z & 0x7fff7fffu, v[i].w & 0x7fff7fffu)));
  mg = max(mg & 0xffffu, mg >> 16);
  int up;
  const float mul = q_factor(mg, up);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t hi[4], lo[4];
    split8(v[2 * i], mul, hi, lo);
    split8(v[2 * i + 1], mul, hi + 2, lo + 2);
    unsigned char* at = q_smem + lane * 128 + ((i ^ (lane & 7)) << 4);
    *reinterpret_cast<uint4*>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(at + kTile * 128) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
  return row_scale_of(P, mul, up);
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(*reinterpret_cast<unsigned long long*>(&d))
      : "l"(*reinterpret_cast<const unsigned long long*>(&a)),
        "l"(*reinterpret_cast<const unsigned long long*>(&b)),
        "l"(*reinterpret_cast<const unsigned long long*>(&c)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(*reinterpret_cast<unsigned long long*>(&d))
      : "l"(*reinterpret_cast<const unsigned long long*>(&a)),
        "l"(*reinterpret_cast<const unsigned long long*>(&b)));
  return d;
}

__device__ __forceinline__ float max3f(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// 32 bytes: a whole sector, so that rows far apart are written without partial ones. p is a multiple
// of 32.
__device__ __forceinline__ void store32(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
               "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// The largest y of 32 columns.
__device__ __forceinline__ float row_max(const uint32_t (&v)[32], const float4* sc, float rs) {
  float mx = -INFINITY;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    float b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = __uint_as_float(v[g * 8 + i]);
    const float t = max3f(max3f(b[0], b[1], b[2]), max3f(b[3], b[4], b[5]), fmaxf(b[6], b[7]));
    mx = fmaxf(mx, fmaf(t, fmaxf(sc[g].x * rs, kTiny), sc[g].y));
  }
  return mx;
}

// P = P1 + P2 of 32 columns, and their part of L. Returned as 8 words of P1, then 8 of P2. A
// masked column is -inf (and its factor is never 0).
__device__ __forceinline__ float weights(const uint32_t (&v)[32], const float4* sc, float rs,
                                         float shift, uint32_t (&o)[16]) {
  float part = 0.f;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const float4 f = sc[g];
    const float k = fmaxf(f.x * rs, kTiny), a = f.y + shift;
    float2 sum = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float2 h[2], l[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int c = g * 8 + 4 * i + 2 * u;
        const float2 x = fma2(make_float2(__uint_as_float(v[c]), __uint_as_float(v[c + 1])),
                              make_float2(k, k), make_float2(a, a));
        const float2 p = make_float2(ex2f(x.x), ex2f(x.y));
        sum = add2(sum, p);
        // to 3 significant bits, and the rest: the last bit of 2^21 p + p is worth a quarter of p's
        // binade, of which 2^21 p is a multiple
        const float2 up = fma2(p, make_float2(2097152.f, 2097152.f), p);
        h[u] = fma2(p, make_float2(-2097152.f, -2097152.f), up);
        l[u] = fma2(h[u], make_float2(-1.f, -1.f), p);
      }
      o[g * 2 + i] = f32_to_e5m2x4(h[0].x, h[0].y, h[1].x, h[1].y);
      o[8 + g * 2 + i] = f32_to_e4m3x4(l[0].x, l[0].y, l[1].x, l[1].y);
    }
    part = fmaf(sum.x + sum.y, f.z, part);
  }
  return part;
}

template <int DP, int NS, int R>
__global__ void __launch_bounds__(kAttThreads, 1)
attend_kernel(const AttendParams P, const __grid_constant__ CUtensorMap k_map,
              const __grid_constant__ CUtensorMap v_map) {
  using L = AttLayout<DP, NS, R>;
  constexpr int SK = L::kKStages, SV = L::kVStages;
  extern __shared__ unsigned char s_raw[];
  unsigned char* smem = s_raw + ((1024 - (smem_u32(s_raw) & 1023)) & 1023);
  AttMisc& m = *reinterpret_cast<AttMisc*>(smem + L::kMisc);
  float4* scales = reinterpret_cast<float4*>(smem + L::kScales);
  const uint32_t base = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* gave_up = &m.gave_up;

  // ---- setup: barriers, tensor memory, this CTA's share of the line of tiles ----
  if (tid < 12) {
    mbar_init(smem_u32(&m.k_full[tid]), 1);
    mbar_init(smem_u32(&m.k_empty[tid]), 1);
    mbar_init(smem_u32(&m.v_full[tid]), 1);
    mbar_init(smem_u32(&m.v_empty[tid]), 1);
  } else if (tid < 14) {
    const int i = tid - 12;
    mbar_init(smem_u32(&m.s_full[i]), 1);
    mbar_init(smem_u32(&m.p_full[i]), 4);
    mbar_init(smem_u32(&m.o_done[i]), 1);
    mbar_init(smem_u32(&m.q_full[i]), NS == 1 && !L::kQTm ? 1 : 4);
    mbar_init(smem_u32(&m.q_empty[i]), NS == 1 ? 9 : 1);
    m.nan_any[i] = 0;
    m.gave_up = 0;
  } else if (tid >= 32 && tid < 32 + kScaleSlots) {
    const int i = tid - 32;
    mbar_init(smem_u32(&m.sc_full[i]), 1);
    mbar_init(smem_u32(&m.sc_empty[i]), NS == 1 ? 4 : 8);
  }
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  if (tid < 256) m.nan_first[tid >> 7][tid & 127] = 0x7fffffff;
  if (warp == 2) tmem_alloc(smem_u32(&m.tmem), 512);
  // What comes before this call on its stream may still be running up to here.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int per = (P.B + kAttThreads - 1) / kAttThreads;
  const int r0 = min(P.B, tid * per), r1 = min(P.B, r0 + per);
  long long mine = 0;
  bool bad = false;
  for (int r = r0; r < r1; ++r) {
    const Request q = request_of(P, r);
    for (int row = 0; row < q.rows; row += L::kRows)
      mine += tiles_for(P, q, min(q.rows, row + L::kRows) - 1) + kUnitCost;
    if (blockIdx.x == 0) bad |= request_bad(P, r);
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
  long long line = 0;  // of one head
  before -= mine;
  for (int w = 0; w < kAttThreads / 32; ++w) {
    if (w < warp) before += m.warp_sum[w];
    line += m.warp_sum[w];
  }
  // Heads outermost: their lines lie one behind another. Where the CTAs divide evenly among them, each
  // head's line is divided for itself: the CTAs at the same place of theirs then read the heads of
  // the same pages at about the same time.
  const int inside = kHeadsInside<NS> ? P.c.Hkv : 1, outside = P.c.Hkv / inside;
  mine *= inside;
  before *= inside;
  line *= inside;
  const int parts = gridDim.x % outside == 0 ? outside : 1, per_part = gridDim.x / parts;
  const long long part = line * (outside / parts);
  const long long share = max((long long)P.min_share, (part + per_part - 1) / per_part);
  const long long p0 = blockIdx.x / per_part * part;
  const long long g0 = p0 + min(part, blockIdx.x % per_part * share), g1 = min(p0 + part, g0 + share);
  if (tid == 0) {
    m.g0 = g0;
    m.share = share;
  }
  const int head0 = line > 0 ? (int)(g0 / line) : 0;
  const long long in_line = g0 - head0 * line;
  if (mine > 0 && g0 < g1 && before <= in_line && in_line < before + mine) {
    long long at = before;
    for (int r = r0; r < r1; ++r) {
      const Request q = request_of(P, r);
      bool found = false;
      for (int row = 0; row < q.rows; row += L::kRows) {
        const int n = tiles_for(P, q, min(q.rows, row + L::kRows) - 1) + kUnitCost;
        if (in_line < at + (long long)n * inside) {
          m.start_item[0] = r;
          m.start_item[1] = row / L::kRows;
          m.start_item[2] = (int)(in_line - at) / n;
          m.start_item[3] = (int)(in_line - at) % n;
          found = true;
          break;
        }
        at += (long long)n * inside;
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

  Schedule<NS, L::kRows> sched;
  sched.g = g0;
  sched.end = g1;
  sched.r = sched.qt = sched.h = sched.off = 0;
  if (g0 < g1) {
    sched.r = m.start_item[0];
    sched.qt = m.start_item[1];
    sched.h = head0 + m.start_item[2];
    sched.off = m.start_item[3];
  }
  Segment s;
  const int log2_bs = P.c.log2_bs, bs = 1 << log2_bs;

  if (warp == 0 || warp == 2) {
    // ---- loads: K by one warp and V by another (a warp takes about 75 cycles to issue a page, 8
    // pages of 16 tokens a tile). Lane p of a tile's pages issues that page; table entries are
    // fetched two batches of tiles ahead and looked at only when they are used ----
    const bool is_v = warp == 2;
    const CUtensorMap* map = is_v ? &v_map : &k_map;
    uint64_t* full = is_v ? m.v_full : m.k_full;
    uint64_t* empty = is_v ? m.v_empty : m.k_empty;
    const int stages = is_v ? SV : SK;
    const int pages = kTile >> log2_bs;                 // of a tile, 1 to 16
    const int batch = 32 / pages < 8 ? 32 / pages : 8;  // tiles whose entries a warp reads at once
    const int my_tile = lane / pages < batch ? lane / pages : -1, my_page = lane % pages;
    const uint32_t dst = base + (is_v ? L::kV : L::kK) + my_page * (uint32_t)(bs * DP);
    int st = 0;
    uint32_t ph = 1;
    bool ok = true;
    while (ok && sched.next(P, s)) {
      const int32_t* table = P.table + (long)s.r * P.max_blocks;
      const int last_page = (s.q.len + bs - 1) >> log2_bs;
      auto entry = [&](int t0) {  // this lane's page of the batch from t0 on; -1: past the context
        const int pg = ((t0 + my_tile) << (7 - log2_bs)) + my_page;
        return my_tile >= 0 && t0 + my_tile < s.b && pg < last_page ? __ldg(table + pg)
                                                                    : P.c.num_blocks;
      };
      int cur = entry(s.a), nxt = entry(s.a + batch);
      for (int t0 = s.a; ok && t0 < s.b; t0 += batch) {
        const int far = entry(t0 + 2 * batch);
        // a page that there is not: beyond the tensor, where the copy fills in zeros
        if ((unsigned)cur >= (unsigned)P.c.num_blocks) {
          if (!is_v && my_tile >= 0 && t0 + my_tile < s.b &&
              ((t0 + my_tile) << (7 - log2_bs)) + my_page < last_page)
            raise_err(P.err, SD_ERR_KV_RANGE);
          cur = P.c.num_blocks;
        }
        for (int j = 0; j < batch && t0 + j < s.b; ++j) {
          const uint32_t bar = smem_u32(full + st);
          ok = mbar_wait_warp(smem_u32(empty + st), ph, gave_up);
          if (!ok) break;
          if (lane == 0) mbar_expect_tx(bar, L::kTileBytes);
          __syncwarp();
          if (my_tile == j)
            tma_load_4d(dst + st * L::kTileBytes, map, 0, s.h, 0, cur, bar);
          if (++st == stages) {
            st = 0;
            ph ^= 1;
          }
        }
        cur = nxt;
        nxt = far;
      }
    }
  } else if (warp == 1) {
    // ---- products: the warp waits, one elected lane issues ----
    constexpr uint32_t hi = desc_hi<DP>();
    constexpr uint32_t qk_idesc = mma_desc(kTile, false, false);
    constexpr uint32_t pv_idesc[2] = {mma_desc(DP, true, true), mma_desc(DP, true, false)};
    const bool lead = elect_one();
    const uint32_t q_lo = desc_lo<DP>(base + L::kQ), k_lo = desc_lo<DP>(base + L::kK),
                   v_lo = desc_lo<DP>(base + L::kV);
    int kst = 0, vst = 0, nq[2] = {0, 0};  // the next unit's first tile in the rings
    uint32_t kph = 0, vph = 0;             // and the parity of its round
    uint32_t pp[2] = {0, 0};
    bool ok = true;
    auto qk = [&](int k_st, int x, int qi) {  // S[x] = Q[qi] K
      if (L::kQTm) {
        const uint32_t d = tmem + x * 128, a = tmem + L::kTmQ + x * 32,
                       k = k_lo + k_st * (L::kTileBytes / 16);
#pragma unroll
        for (int term = 0; term < 2; ++term)
#pragma unroll
          for (int kk = 0; kk < DP / 32; ++kk)
            mma_ts<hi, qk_idesc>(d, a + term * 16 + kk * 8, k + kk * 2, term + kk > 0);
        return;
      }
      const uint32_t d = tmem + x * 128, a = q_lo + qi * (2 * L::kQBytes / 16),
                     k = k_lo + k_st * (L::kTileBytes / 16);
#pragma unroll
      for (int term = 0; term < 2; ++term)
#pragma unroll
        for (int kk = 0; kk < DP / 32; ++kk)
          mma_ss<hi, qk_idesc>(d, a + term * (L::kQBytes / 16) + kk * 2, k + kk * 2,
                               term + kk > 0);
    };
    auto pv = [&](int v_st, int x, bool add) {  // O[x] += P V
      const uint32_t d = tmem + L::kTmO + x * DP, a = tmem + x * 128,
                     v = v_lo + v_st * (L::kTileBytes / 16);
#pragma unroll
      for (int kk = 0; kk < kTile / 32; ++kk) {
        mma_ts<hi, pv_idesc[0]>(d, a + kk * 16, v + kk * (32 * DP / 16), add || kk > 0);
        mma_ts<hi, pv_idesc[1]>(d, a + kk * 16 + 8, v + kk * (32 * DP / 16), true);
      }
    };
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      ok = ok && mbar_wait_warp(smem_u32(bar), parity, gave_up);
      return ok;
    };
    while (ok && sched.next(P, s)) {
      const int T = s.b - s.a;
      if (NS == 1) {
        const int qb = nq[0] & 1;  // units alternate between two buffers
        bool q_there[2] = {!L::kQTm, !L::kQTm};
        if (!L::kQTm) {
          if (!wait(&m.q_full[qb], (nq[0] >> 1) & 1)) break;
          ++nq[0];
        }
        // Each stream has its own place in the rings. Whatever is ready is issued: a stream's PV
        // once its P is there, its next QK once P, in the place of S, is used.
        int kj[2] = {0, 1}, vj[2] = {0, 1}, ks[2], vs[2];
        uint32_t kp[2], vp[2];
        bool s_free[2] = {true, true};
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          ks[x] = kst + x;
          kp[x] = kph;
          if (ks[x] >= SK) {
            ks[x] -= SK;
            kp[x] ^= 1;
          }
          vs[x] = vst + x;
          vp[x] = vph;
          if (vs[x] >= SV) {
            vs[x] -= SV;
            vp[x] ^= 1;
          }
        }
        long long idle = 0;  // the clock when nothing was ready first
        while (vj[0] < T || vj[1] < T) {
          bool did = false;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (vj[x] < T && mbar_test_warp(smem_u32(&m.p_full[x]), pp[x])) {
              if (!wait(&m.v_full[vs[x]], vp[x])) break;
              pp[x] ^= 1;
              tc_fence_after();
              if (lead) {
                pv(vs[x], x, vj[x] >= 2);
                mma_commit(smem_u32(&m.o_done[x]));
                mma_commit(smem_u32(&m.v_empty[vs[x]]));
              }
              s_free[x] = true;
              vj[x] += 2;
              vs[x] += 2;
              if (vs[x] >= SV) {
                vs[x] -= SV;
                vp[x] ^= 1;
              }
              did = true;
            }
            if (L::kQTm && !q_there[x] && kj[x] < T &&
                mbar_test_warp(smem_u32(&m.q_full[x]), nq[x] & 1)) {
              ++nq[x];
              q_there[x] = true;
            }
            // (the parity of a phase means something only once the phase before has been seen to end;
            // with an odd number of stages that one was the other stream's)
            if (q_there[x] && s_free[x] && kj[x] < T &&
                (SK % 2 == 0 || kj[x] - kj[x ^ 1] < SK) &&
                mbar_test_warp(smem_u32(&m.k_full[ks[x]]), kp[x])) {
              tc_fence_after();
              if (lead) {
                qk(ks[x], x, qb);
                mma_commit(smem_u32(&m.s_full[x]));
                mma_commit(smem_u32(&m.k_empty[ks[x]]));
                if (!L::kQTm && kj[x] + 2 >= T && kj[x ^ 1] >= T)
                  mma_commit(smem_u32(&m.q_empty[qb]));
              }
              s_free[x] = false;
              kj[x] += 2;
              ks[x] += 2;
              if (ks[x] >= SK) {
                ks[x] -= SK;
                kp[x] ^= 1;
              }
              did = true;
            }
          }
          if (!ok) break;
          if (did) {
            idle = 0;
          } else {
            const long long now = clock64();
            if (idle == 0) idle = now;
            // (lane 0's clock decides for the warp)
            if (__shfl_sync(0xffffffffu, (int)(now - idle > kWaitClocks || *gave_up), 0)) {
              *gave_up = 1;
              ok = false;
              break;
            }
          }
        }
        kst += T % SK;
        kph ^= (T / SK) & 1;
        if (kst >= SK) {
          kst -= SK;
          kph ^= 1;
        }
        vst += T % SV;
        vph ^= (T / SV) & 1;
        if (vst >= SV) {
          vst -= SV;
          vph ^= 1;
        }
      } else {
#pragma unroll
        for (int x = 0; x < 2; ++x)
          if ((x ? s.cnt1 : s.cnt0) > 0) wait(&m.q_full[x], nq[x]++ & 1);
        auto do_qk = [&](int j, int x) {
          if (!wait(&m.k_full[kst], kph)) return;
          tc_fence_after();
          if (lead) {
            qk(kst, x, x);
            mma_commit(smem_u32(&m.s_full[x]));
            if (!L::kQTm && j == (x ? s.cnt1 : s.cnt0) - 1)
              mma_commit(smem_u32(&m.q_empty[x]));
          }
        };
        auto k_done = [&] {
          if (ok && lead) mma_commit(smem_u32(&m.k_empty[kst]));
          if (++kst == SK) {
            kst = 0;
            kph ^= 1;
          }
        };
#pragma unroll
        for (int x = 0; x < 2; ++x)
          if ((x ? s.cnt1 : s.cnt0) > 0) do_qk(0, x);
        k_done();
        for (int j = 0; ok && j < T; ++j) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int cnt = x ? s.cnt1 : s.cnt0;
            if (j >= cnt) continue;
            wait(&m.p_full[x], pp[x]);
            if (!wait(&m.v_full[vst], vph)) break;
            pp[x] ^= 1;
            tc_fence_after();
            if (lead) {
              pv(vst, x, j > 0);
              if (x == 1 || j >= s.cnt1) mma_commit(smem_u32(&m.v_empty[vst]));
              mma_commit(smem_u32(&m.o_done[x]));
            }
            if (j + 1 < cnt) do_qk(j + 1, x);
          }
          if (j + 1 < T) k_done();
          if (++vst == SV) {
            vst = 0;
            vph ^= 1;
          }
        }
      }
    }
    __syncwarp();
  } else if (warp == 3) {
    // ---- Q of the next unit while this one is computed, and the scales: 16 entries a tile, one
    // for 8 tokens, two tiles at a time; table entries two passes and scales one pass ahead ----
    const int e = lane & 15, half = lane >> 4;
    int nq = 0, slot = 0;
    uint32_t sc_ph = 1;
    bool ok = true;
    while (ok && sched.next(P, s)) {
      const int32_t* table = P.table + (long)s.r * P.max_blocks;
      auto entry = [&](int t0) {
        const long tok = (long)(t0 + half) * kTile + e * 8;
        return t0 + half < s.b && tok < s.q.len ? __ldg(table + (tok >> log2_bs)) : -1;
      };
      auto scales_of = [&](int page) {  // (K's, V's; -1: no page)
        if ((unsigned)page >= (unsigned)P.c.num_blocks) return make_float2(0.f, -1.f);
        const long at = (long)page * P.c.Hkv + s.h;
        return make_float2(__ldg(P.c.k_scale + at), __ldg(P.c.v_scale + at));
      };
      int nxt = entry(s.a + 2);
      float2 sc = scales_of(entry(s.a));
      if (NS == 1 && !L::kQTm) {
        const int qb = nq & 1;
        ok = mbar_wait_warp(smem_u32(&m.q_empty[qb]), ((nq >> 1) & 1) ^ 1, gave_up);
        if (!ok) break;
        load_q<DP, R, 32>(P, s, s.row0, s.rows, smem + L::kQ + qb * 2 * L::kQBytes,
                          m.row_scale + qb * kTile, lane);
        fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&m.q_full[qb]));
        ++nq;
      }
      for (int t0 = s.a; ok && t0 < s.b; t0 += 2) {
        const int far = entry(t0 + 4);
        const float2 sc_nxt = scales_of(nxt);
        const bool none = sc.y == -1.f, zero = !none && !(sc.y > 0.f) && sc.y == sc.y;
        // (a NaN stays out of here; the approximations are exact for powers of two, and off by 2^-22 of
        // a weight at most for others)
        const float v = fmaxf(sc.y, kMinScale);
        const float4 f = make_float4(
            sc.x, none ? -INFINITY : zero ? kZeroLog2 : sc.y != sc.y ? sc.y : __log2f(v),
            none ? 1.f : zero ? kZeroInv : __fdividef(1.f, v), 0.f);
        const uint32_t zeros = __ballot_sync(0xffffffffu, zero);
        const uint32_t k_zeros = __ballot_sync(0xffffffffu, !none && sc.x == 0.f);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if (t0 + k >= s.b) break;
          ok = mbar_wait_warp(smem_u32(&m.sc_empty[slot]), sc_ph, gave_up);
          if (!ok) break;
          if (half == k) scales[slot * 16 + e] = f;
          if (lane == 0)
            m.sc_zero[slot] = k ? zeros >> 16 | (k_zeros & 0xffff0000u)
                                : (zeros & 0xffffu) | k_zeros << 16;
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&m.sc_full[slot]));
          if (++slot == kScaleSlots) {
            slot = 0;
            sc_ph ^= 1;
          }
        }
        nxt = far;
        sc = sc_nxt;
      }
    }
  }
  if (warp >= 4) {
    // ---- softmax: stream x, one row a thread ----
    constexpr int NC = 4 / R;                             // 32-column chunks of a thread
    const int x = (warp - 4) >> 2, wt = tid - 128 - x * 128;  // thread of its stream
    const int quarter = warp & 3;                             // of the lanes
    const int copy = quarter / NC;                            // which columns: chunks copy*NC..
    const int wr = (quarter % NC) * 32 + lane;                // row of this thread in its tile
    const uint32_t lanes = (uint32_t)quarter << 21;
    const uint32_t tS = tmem + x * 128 + lanes;
    const uint32_t tO0 = tmem + L::kTmO + lanes, tO = tO0 + x * DP;  // the first's, this stream's
    // A wait for V is for this tile's phase only if the one before in the same stage is known to have
    // ended. With an odd number of stages that one was the other stream's: S of this tile, which
    // comes after that stream's product with it, has to be there. Else it was this stream's own.
    // (Waiting for S first everywhere: 64 requests 129 instead of 122 us, a prompt 650 instead of 640.)
    constexpr bool kSFirst = NS == 1 && SV % 2 == 1;
    // The accumulator is rescaled before P is formed (heads of 64), or after, when S's registers are
    // free and 64 columns go at a time. Before against after: 64 requests 122 to 126 us, drafter batch
    // 413 to 411, 256 requests 899 to 889, prompt 664 to 640.
    constexpr bool kLate = DP == 128;
    int it = 0, nq = 0, unit = 0;
    int done = 0;  // tiles of this stream so far
    bool ok = true;
    bool continues = false;
    JoinDesc jd;
    jd.pieces = 0;
    // Every thread passes every named barrier, also once a wait has run out (ok is false then, and
    // nothing is computed any more).
    while (sched.next(P, s)) {
      const int T = s.b - s.a;
      const int cnt_x = x ? s.cnt1 : s.cnt0;
      const int buf = unit & 1;
      const int row_base = NS == 1 ? 0 : x * kTile;       // of this stream in the unit
      const int my_rows = NS == 1 ? s.rows : min(kTile, s.rows - row_base);
      float rs = 0.f;
      const int row = s.row0 + row_base + wr;
      const bool warp_live = (quarter % NC) * 32 < my_rows;
      const bool live = wr < my_rows;
      // 1. Q (but for one Q tile in shared memory, loaded here), and this row's scale
      if (L::kQTm) {
        if (cnt_x > 0) {  // (every product of this stream's last unit is done)
          if (ok && warp_live) rs = q_to_tmem(P, s, row, live, tmem + L::kTmQ + x * 32 + lanes);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&m.q_full[x]));
        }
      } else if (NS == 1) {
        ok = ok && mbar_wait_warp(smem_u32(&m.q_full[unit & 1]), (unit >> 1) & 1, gave_up);
        rs = m.row_scale[(unit & 1) * kTile + wr];
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&m.q_empty[unit & 1]));
      } else if (cnt_x > 0) {
        ok = ok && mbar_wait_warp(smem_u32(&m.q_empty[x]), (nq & 1) ^ 1, gave_up);
        ++nq;
        if (ok && warp_live)
          rs = q_to_smem(P, s, row, live, wt, smem + L::kQ + x * 2 * L::kQBytes);
        fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&m.q_full[x]));
      }
      const int lim = seen_by(P, s.q, min(row, s.row0 + s.rows - 1));
      const int min_lim = seen_by(P, s.q, s.row0 + row_base);
      float M = -INFINITY, Lsum = 0.f;
      m.ml[x][wt].x = -INFINITY;  // (every reader of the last unit's has passed its barrier)

      // 2. tiles
      for (int j = NS == 1 ? x : 0; ok && j < T; j += NS == 1 ? 2 : 1) {
        const int slot = (it + j) % kScaleSlots;
        ok = mbar_wait_warp(smem_u32(&m.sc_full[slot]), ((it + j) / kScaleSlots) & 1, gave_up);
        if (!ok) break;
        if (NS == 2 && j >= cnt_x) {  // the other stream's alone
          if (lane == 0) mbar_arrive(smem_u32(&m.sc_empty[slot]));
          continue;
        }
        const int t0 = (s.a + j) * kTile;
        const uint32_t zero = m.sc_zero[slot] & 0xffffu, k_zero = m.sc_zero[slot] >> 16;
        const bool masked = t0 + kTile > min_lim;
        if (kSFirst) {
          ok = mbar_wait_warp(smem_u32(&m.s_full[x]), done & 1, gave_up);
          if (!ok) break;
          tc_fence_after();
        }
        if (masked || zero) {
          // V's rows that no row of this call sees become 0, and NaN among the others too (they
          // are noted, for the rows that see them): 0 times NaN is no 0
          const int st = (it + j) % SV;
          ok = mbar_wait_warp(smem_u32(&m.v_full[st]), ((it + j) / SV) & 1, gave_up);
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
        if (!kSFirst) {
          ok = mbar_wait_warp(smem_u32(&m.s_full[x]), done & 1, gave_up);
          if (!ok) break;
          tc_fence_after();
        }
        if (warp_live) {
          const float4* sc = scales + slot * 16 + copy * NC * 4;
          const int edge = lim - t0 - copy * NC * 32;  // columns from here on are masked
          const uint32_t tC = tS + copy * NC * 32;
          // rare: where they lie, the masked columns of S become -inf, and those of pages whose K is
          // zeros 0, whatever the bytes (but for a row whose queries make every score NaN)
          if (masked || k_zero) {
#pragma unroll 1
            for (int c = 0; c < NC; ++c) {
              uint32_t v[32];
              tmem_ld32(tC + c * 32, v);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                if ((k_zero >> ((copy * NC + c) * 4 + i / 8)) & 1 && rs == rs) v[i] = 0;
                v[i] = c * 32 + i >= edge ? 0xff800000u : v[i];
              }
              __syncwarp();
              tmem_st32(tC + c * 32, v);
            }
            tmem_wait_st();
          }
          // Up to 64 columns of S stay in registers; of 128, 32 at a time are read, twice, the next
          // ones on their way. (The code of one pass stays small for the instruction cache, which
          // eight warps share.)
          uint32_t v[32], w[32];
          float mx = -INFINITY;
          tmem_ld32(tC, v);
          if (NC == 2) tmem_ld32(tC + 32, w);
          tmem_wait_ld();
          if (NC <= 2) {
            mx = row_max(v, sc, rs);
            if (NC == 2) mx = fmaxf(mx, row_max(w, sc + 4, rs));
          } else {
#pragma unroll 1
            for (int c = 0; c < NC; c += 2) {
              tmem_ld32(tC + (c + 1) * 32, w);
              mx = fmaxf(mx, row_max(v, sc + c * 4, rs));
              tmem_wait_ld();
              tmem_ld32(tC + (c + 2 < NC ? c + 2 : 0) * 32, v);
              mx = fmaxf(mx, row_max(w, sc + c * 4 + 4, rs));
              tmem_wait_ld();
            }
          }
          const bool fall = mx < M - kFall && mx > -INFINITY;
          const bool rise = mx > M + kSlack;
          const bool moved = __any_sync(0xffffffffu, rise || fall);
          float fac = 1.f;
          if (moved) {  // (a row's own y alone decide on its reference)
            const float top = m.ml[x][wt].x;
            float Mn = fall ? fmaxf(mx + kAbove, top - kDeepest) : rise ? mx : M;
            if (fall && !(Lsum * ex2f(M - Mn) < kMaxL)) Mn = M;
            m.ml[x][wt].x = fmaxf(top, Mn);
            fac = M == -INFINITY ? 0.f : ex2f(M - Mn);
            Lsum *= fac;
            M = Mn;
          }
          // The accumulator's old sums in the new reference's units.
          auto rescale = [&] {
            if (!moved || j < (NS == 1 ? 2 : 1)) return;
            ok = mbar_wait_warp(smem_u32(&m.o_done[x]), (done - 1) & 1, gave_up);
            if (!ok) return;
            tc_fence_after();
            constexpr int kStep = kLate ? 2 : 1;
#pragma unroll 1
            for (int c = 0; c < DP; c += 32 * kStep) {
              uint32_t u[kStep][32];
#pragma unroll
              for (int k = 0; k < kStep; ++k) tmem_ld32(tO + c + k * 32, u[k]);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < kStep; ++k) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  u[k][i] = __float_as_uint(__uint_as_float(u[k][i]) * fac);
                tmem_st32(tO + c + k * 32, u[k]);
              }
            }
          };
          if (!kLate) rescale();
          if (!ok) break;
          const float shift = kShift - (M == -INFINITY ? 0.f : M);
          uint32_t o[16];
          if (NC <= 2) {
            Lsum += weights(v, sc, rs, shift, o);
            tmem_st16(tS + copy * NC * 16, o);
            if (NC == 2) {
              Lsum += weights(w, sc + 4, rs, shift, o);
              tmem_st16(tS + (copy * NC + 1) * 16, o);
            }
          } else {
#pragma unroll 1
            for (int c = 0; c < NC; c += 2) {
              tmem_ld32(tC + (c + 1) * 32, w);
              Lsum += weights(v, sc + c * 4, rs, shift, o);
              tmem_wait_ld();
              tmem_st16(tS + c * 16, o);
              if (c + 2 < NC) tmem_ld32(tC + (c + 2) * 32, v);
              Lsum += weights(w, sc + c * 4 + 4, rs, shift, o);
              tmem_wait_ld();
              tmem_st16(tS + (c + 1) * 16, o);
            }
          }
          if (kLate) rescale();
          if (!ok) break;
          if (R > 1) {  // the other copies' columns count as zero here
            const uint32_t none[16] = {};
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (c / NC != copy) tmem_st16(tS + c * 16, none);
          }
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&m.sc_empty[slot]));
          mbar_arrive(smem_u32(&m.p_full[x]));
        }
        ++done;
      }

      // 3. the unit's (or this part's) result
      const bool split = s.a > 0 || s.b < s.n;
      const int cnt_b = NS == 1 ? s.cnt1 : 0;
      if (NS == 1) {
        // (each stream waits for its own products, the barrier joins the two: the parity of the other
        // stream's says nothing here, it may be two phases behind. A stream's count goes on from
        // unit to unit; one without a tile has no phase to wait for)
        if (x == 0 || cnt_b > 0)
          ok = ok && mbar_wait_warp(smem_u32(&m.o_done[x]), (done - 1) & 1, gave_up);
        m.ml[x][wt] = make_float2(M, Lsum);
      } else if (cnt_x > 0) {
        ok = ok && mbar_wait_warp(smem_u32(&m.o_done[x]), (done - 1) & 1, gave_up);
      }
      tc_fence_before();
      named_bar(1, 256);
      tc_fence_after();
      const bool has_nan = m.nan_any[buf] != 0;
      if (tid - 128 < 128) m.nan_first[buf ^ 1][tid - 128] = 0x7fffffff;
      if (tid == 128) m.nan_any[buf ^ 1] = 0;
      float* slot = slots + (2L * blockIdx.x + (s.a > 0 ? 0 : 1)) * L::kSlotFloats;
      const int* nan_first = m.nan_first[buf];
      if (R > 1) {
        // 2R partial rows: every warp leaves some columns of its own, weighed by their common
        // maximum, then the threads add them up in the warps' order
        float* join = reinterpret_cast<float*>(smem + L::kJoin);
        constexpr int parts = 2 * R;  // a stream without a tile counts with weight 0
        float Mt = -INFINITY, Lt = 0.f;
        float2 ml[parts];
#pragma unroll
        for (int i = 0; i < parts; ++i) {
          ml[i] = m.ml[i / R][(i % R) * (kTile / R) + wr];
          Mt = fmaxf(Mt, ml[i].x);
        }
#pragma unroll
        for (int i = 0; i < parts; ++i)
          Lt += ml[i].y * (ml[i].x == Mt ? 1.f : ex2f(ml[i].x - Mt));
        const float inv = Lt == 0.f ? 0.f : 1.f / Lt;
        const float lse2 = Lt == 0.f ? -INFINITY : Mt - kShift + log2f(Lt);
        const float wm = (M == Mt ? 1.f : ex2f(M - Mt)) * inv;
        const bool used = x == 0 || cnt_b > 0;
        if (ok && x == 0 && copy == 0 && live) {
          if (split) slot[(long)L::kRows * DP + wr] = lse2;
          else if (P.lse) {
            const int2 th = token_head(P, row);
            P.lse[(long)(s.q.tok0 + th.x) * P.Hq + s.h * P.G + th.y] = lse2 * kLn2F;
          }
        }
        constexpr int kJC = L::kJoinCols;
#pragma unroll 1
        for (int c = 0; c < DP; c += kJC) {
          __syncwarp();
          if (ok && warp_live) {
            float* mine = join + ((warp - 4) * 32 + lane) * (kJC + 1);
#pragma unroll
            for (int k = 0; k < kJC; k += 16) {
              uint32_t u[16];
              tmem_ld16(tO + c + k, u);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i)
                mine[k + i] = used ? __uint_as_float(u[i]) * wm : 0.f;
            }
          }
          named_bar(1, 256);
          // 4 columns a thread
          const int cc = ((tid - 128) % (kJC / 4)) * 4;
          for (int r = (tid - 128) / (kJC / 4); ok && r < s.rows; r += 1024 / kJC) {
            float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < parts; ++i) {
              const int w = (i / R) * 4 + (i % R) * NC + (r >> 5);
              const float* from = join + (w * 32 + (r & 31)) * (kJC + 1) + cc;
#pragma unroll
              for (int k = 0; k < 4; ++k) o[k] += from[k];
            }
            const int rr = s.row0 + r;
            if (has_nan) {
              const int l = seen_by(P, s.q, rr);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (nan_first[c + cc + k] < l) o[k] = nanf("");
            }
            if (split) {
              *reinterpret_cast<float4*>(slot + (long)r * DP + c + cc) =
                  make_float4(o[0], o[1], o[2], o[3]);
            } else if (c + cc < P.c.D) {
              const __nv_bfloat162 a = __floats2bfloat162_rn(o[0], o[1]);
              const __nv_bfloat162 b = __floats2bfloat162_rn(o[2], o[3]);
              const int2 th = token_head(P, rr);
              *reinterpret_cast<uint2*>(P.out + (long)(s.q.tok0 + th.x) * P.ld_out +
                                        (long)(s.h * P.G + th.y) * P.hs_out + c + cc) =
                  make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                             *reinterpret_cast<const uint32_t*>(&b));
            }
          }
          if (c + kJC < DP) named_bar(1, 256);
        }
      } else {
        float wa = 1.f, wb = 0.f, Mt = M, Lt = Lsum;
        if (NS == 1) {
          const float2 a = m.ml[0][wt], b = m.ml[1][wt];
          Mt = a.x;
          Lt = a.y;
          if (cnt_b > 0) {
            Mt = fmaxf(a.x, b.x);
            wa = a.x == Mt ? 1.f : ex2f(a.x - Mt);
            wb = b.x == Mt ? 1.f : ex2f(b.x - Mt);
            Lt = a.y * wa + b.y * wb;
          }
        }
        const float inv = Lt == 0.f ? 0.f : 1.f / Lt;
        const float lse2 = Lt == 0.f ? -INFINITY : Mt - kShift + log2f(Lt);
        wa *= inv;
        wb *= inv;
        const int unit_row = row_base + wt;
        const int2 th = token_head(P, row);
        const long tok = s.q.tok0 + th.x;
        const int hq = s.h * P.G + th.y;
        const bool mine_any = NS == 1 || cnt_x > 0;
        if (ok && warp_live && my_rows > 0) {
          constexpr int kCols = NS == 1 ? DP / 2 : DP;  // this thread's share of the row
          const int c0 = NS == 1 ? x * kCols : 0;
          if (mine_any) {
#pragma unroll 1
            for (int c = 0; c < kCols; c += 32) {
              __syncwarp();  // (a partial warp's lanes without a row come back here)
              uint32_t u[32], w[32];
              tmem_ld32((NS == 1 ? tO0 : tO) + c0 + c, u);
              if (NS == 1 && cnt_b > 0) tmem_ld32(tO0 + DP + c0 + c, w);
              tmem_wait_ld();
              float o[32];
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                o[i] = __uint_as_float(u[i]) * wa;
                if (NS == 1 && cnt_b > 0) o[i] = fmaf(__uint_as_float(w[i]), wb, o[i]);
              }
              if (has_nan) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  if (nan_first[c0 + c + i] < lim) o[i] = nanf("");
              }
              if (!live) {
              } else if (split) {
                float* p = slot + (long)unit_row * DP + c0 + c;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  store32(p + i * 8, reinterpret_cast<const uint32_t*>(o + i * 8));
              } else {
                uint16_t* p = P.out + tok * P.ld_out + hq * P.hs_out + c0 + c;
                uint32_t b[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  const __nv_bfloat162 h2 = __floats2bfloat162_rn(o[2 * i], o[2 * i + 1]);
                  b[i] = *reinterpret_cast<const uint32_t*>(&h2);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  if (c0 + c + i * 16 >= P.c.D) break;  // D is a multiple of 16
                  if (P.out_32) {
                    store32(p + i * 16, b + i * 8);
                  } else {
                    uint4* q4 = reinterpret_cast<uint4*>(p + i * 16);
                    q4[0] = make_uint4(b[i * 8], b[i * 8 + 1], b[i * 8 + 2], b[i * 8 + 3]);
                    q4[1] = make_uint4(b[i * 8 + 4], b[i * 8 + 5], b[i * 8 + 6], b[i * 8 + 7]);
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
      }
      if (s.a == 0 && s.b < s.n) {  // begun here, ended by a later CTA
        continues = true;
        // (the last tile's place over the share, counted from this CTA's)
        jd.pieces = (int)((s.first + s.n - 1 - m.g0) / m.share + 1);
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
  if (warp == 2) tmem_free(tmem, 512);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Joins the parts of a unit that several CTAs shared: one warp a row, parts in their order.
template <int DP, int NS, int R>
__global__ void __launch_bounds__(256) attend_join_kernel(const AttendParams P) {
  using L = AttLayout<DP, NS, R>;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
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
  const int2 th = token_head(P, d.row0 + r);
  const long tok = d.tok0 + th.x;
  const int hq = d.head * P.G + th.y;
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
  static std::atomic<int> count[64];  // (threads that come first together all find the same)
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  int n = count[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    count[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

template <int DP, int NS, int R>
static int launch_attend(const AttendParams& P, const CUtensorMap& km, const CUtensorMap& vm,
                         int ctas, bool join, cudaStream_t stream) {
  using L = AttLayout<DP, NS, R>;
  constexpr int smem = L::kMisc + (int)sizeof(AttMisc) + 1024;
  static_assert(smem <= 227 * 1024, "shared memory of one CTA");
  static std::atomic<bool> set[64];  // per device; true only once the attribute is in force
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return SD_E_DEVICE;
  if (!set[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(attend_kernel<DP, NS, R>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             smem) != cudaSuccess)
      return SD_E_LAUNCH;
    set[dev].store(true, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas, 1, 1);
  cfg.blockDim = dim3(kAttThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, attend_kernel<DP, NS, R>, P, km, vm) != cudaSuccess)
    return SD_E_LAUNCH;
  if (!join) return SD_OK;
  cudaLaunchConfig_t jc = {};
  jc.gridDim = dim3((unsigned)ctas, (unsigned)(L::kRows / 8), 1);
  jc.blockDim = dim3(256, 1, 1);
  jc.stream = stream;
  jc.attrs = attr;
  jc.numAttrs = 1;
  return cudaLaunchKernelEx(&jc, attend_join_kernel<DP, NS, R>, P) == cudaSuccess ? SD_OK
                                                                               : SD_E_LAUNCH;
}

}  // namespace sdk

extern "C" size_t sd_kv_attend_workspace_launch(int D) {
  const long slot = D <= 64 ? sdk::AttLayout<64, 2, 1>::kSlotFloats
                            : sdk::AttLayout<128, 2, 1>::kSlotFloats;
  // (16 bytes to begin at a multiple of 32)
  return 16 + sdk::kMaxCtas * sizeof(sdk::JoinDesc) +
         (size_t)2 * sdk::kMaxCtas * slot * sizeof(float);
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
  P.g_magic = P.G > 1 ? ~0ull / (unsigned)P.G + 1 : 0;
  P.scale = sm_scale * sdk::kLog2eF;
  P.out = (uint16_t*)out;
  P.ld_out = ld_out;
  P.hs_out = hs_out;
  P.lse = lse;
  P.out_32 = (uintptr_t)out % 32 == 0 && ld_out % 16 == 0 && hs_out % 16 == 0;
  // store32 needs every part of a row at a multiple of 32; the caller's scratch is at one of 16
  static_assert(sizeof(sdk::JoinDesc) % 32 == 0, "the parts begin at a multiple of 32");
  P.ws = (unsigned char*)(((uintptr_t)workspace + 31) / 32 * 32);
  P.err = err;
  // A CTA's least share: a unit's cost and 4 tiles. With 1, 4 and 16 tiles one token at 500 tokens
  // takes 16.3, 15.7, 15.7 us, at 1000 19.6, 16.9, 19.2, at 4000 19.6, 21.5, 26.1.
  P.min_share = sdk::kUnitCost + 4;
  const int sms = sdk::sm_count();
  if (sms < 1) return SD_E_DEVICE;
  const int ctas = sms < sdk::kMaxCtas ? sms : sdk::kMaxCtas;
  CUtensorMap km, vm;
  const int DP = D <= 64 ? 64 : 128;
  if (!sdk::cache_map(&km, k_cache, P.c, DP) || !sdk::cache_map(&vm, v_cache, P.c, DP))
    return SD_E_SHAPE;
  // units of one tile are never shared
  const bool join = ((long)max_blocks << log2_bs) > sdk::kTile;
  // The expected rows of a request choose the unit: 32 or 64 rows stand in the lanes four times or
  // twice, so that all softmax warps share a tile's columns; more than 128 make two Q tiles. Measured
  // in us with units of 32, 64, 128 and 256 rows: heads of 64, 64 requests of 32 rows 102, 104, 148,
  // 201; 48 rows 195, 118, 160, 219; 96 rows 279, 206, 161, 214; 192 rows 605, 351, 336, 297. Heads of
  // 128, 256 requests of 32 rows 887, 923, 1184, 1877; 56 rows 1700, 950, 1262, 1845; 112 rows 3711,
  // 1947, 1404, 1957; 64 requests of 240 rows 1788, 988, 749, 610.
  const long rows = (long)max_q * P.G;
  if (DP == 64) {
    if (rows <= 32) return sdk::launch_attend<64, 1, 4>(P, km, vm, ctas, join, stream);
    if (rows <= 64) return sdk::launch_attend<64, 1, 2>(P, km, vm, ctas, join, stream);
    if (rows <= 128) return sdk::launch_attend<64, 1, 1>(P, km, vm, ctas, join, stream);
    return sdk::launch_attend<64, 2, 1>(P, km, vm, ctas, join, stream);
  }
  if (rows <= 32) return sdk::launch_attend<128, 1, 4>(P, km, vm, ctas, join, stream);
  if (rows <= 64) return sdk::launch_attend<128, 1, 2>(P, km, vm, ctas, join, stream);
  if (rows <= 128) return sdk::launch_attend<128, 1, 1>(P, km, vm, ctas, join, stream);
  return sdk::launch_attend<128, 2, 1>(P, km, vm, ctas, join, stream);
}
