// Attention of a generation step for a batch that shares a long prefix: every
// request's queries see the prefix's keys, kept once for all of them, and the
// keys of the request's own cache, whose length only the device knows.
//
// For request b with own length n, query row i (of Lq) sits at position
// a = P + n - Lq + i behind the P prefix keys and sees the keys j <= a of
// [prefix; own cache] with a - j < W (W = 0: all of them).  A softmax over two
// key sets splits exactly: each set (and each part of one) gives its maximum
// m, its sum l of 2^(s - m) and its unnormalised O, and with M = max m
//   o = sum 2^(m - M) O / sum 2^(m - M) l,   lse = (M + log2 sum 2^(m - M) l) ln 2.
//
// Work.  The unit is one key tile (T = 128 keys) of one segment.  A segment is
// the product of one block of query rows with one kv head's prefix (up to N
// rows, packed from as many requests as fit, so the prefix is read once for
// all of them), or with one request's own cache (up to 16 rows: the G * Lq
// rows of a kv head).  One CTA per SM works first on pieces of the prefix,
// then on a run of the requests' own tiles, sized so that all CTAs get the
// same number of units however ragged the lengths are: every CTA sums the
// device-side lengths itself, no host sees them, and no counter has to be
// reset between calls.  The pieces of one key range with all its row blocks
// are neighbouring CTAs' work at the same time, so a tile's second and later
// reads find it in L2.  Each piece, and each CTA's share of an own segment,
// leaves one partial (m, l, O) in a slot of its own; a second kernel merges a
// row's partials.
//
// Products are transposed, as in the decode kernel: S^T (128 keys x N rows) =
// K_tile Q^T and O^T (D x N rows) += V_tile^T P^T, so the keys fill the MMA's
// M dimension whatever the number of query rows is.  K, V and q are read as
// bf16, and P is rounded to bf16 for the second product (both operands of an
// MMA have one type; o itself is bf16).  S, l, m and O are fp32.
//
// Own tiles are aligned to the cache's end: a tile that would reach past it
// starts earlier (below key 0 the TMA fills zeros), so whatever the cache
// holds behind a request's length is never loaded.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "swa_internal.h"
#include "tc_ptx.cuh"

namespace swa {
namespace {

using namespace tc;

constexpr int T = 128;      // keys per tile
constexpr int kOwnRows = 16;  // query rows of an own segment (MMA N)
constexpr int kSMs = 152;   // one CTA per SM
constexpr int kPieces = 2 * kSMs;  // prefix pieces (or as many as there are segments)
constexpr int kSmemMax = 232448;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// P, its sums and O are bf16 and fp32, whose exponents reach 2^127: a row's
// reference maximum (that of its first tile with a visible key) only moves
// when a score outgrows it by more than 2^32, which leaves 2^63 for the sum
// over 2^31 keys and loses no bit, since their precision is relative.
constexpr float kGrowLog2 = 32.0f;
// plan words: prefix tiles, ranges of a prefix segment, the own runs (four
// words), then from kPlanOff on each request's first own tile
constexpr int kPlanOff = 8;

struct SharedParams {
  SharedGeom g;
  SharedSplit s;
  const int* own_len;
  const float* sinks;  // [Hq] or null
  uint16_t* o;         // bf16 [B, Hq, Lq, D]
  float* lse;          // [B, Hq, Lq]
  int* plan;
  float *pp_ml, *pp_o;  // prefix partials: [piece][rows][2] and [piece][rows][D]
  float *po_ml, *po_o;  // own partials: [slot][rows]...
  int* status;
};

// The tiles of a request's own cache that any of its rows sees; a negative
// length is an empty place of the batch.
__device__ __forceinline__ int own_tiles(const SharedGeom& g, int len) {
  const int n = min(len, g.own_rows);
  const int lo = g.W > 0 ? max(0, n - g.Lq - g.W + 1) : 0;
  return n > lo ? (n - lo + T - 1) / T : 0;
}

// The CTAs' runs of own units: `rich` CTAs with qa each, then the others with
// qb each; the last CTA's ends with the units.
struct OwnRuns {
  int rich, qa, qb, units;
  __device__ __forceinline__ int start(int c) const {
    const long long u = c < rich ? (long long)c * qa : (long long)rich * qa + (long long)(c - rich) * qb;
    return c >= kSMs || u > units ? units : (int)u;
  }
  __device__ __forceinline__ int owner(int u) const {  // of unit u < units
    const long long r = (long long)rich * qa;
    return u < r ? u / qa : min(rich + (int)(u - r) / qb, kSMs - 1);
  }
};

// A place in a CTA's prefix pieces.  Piece p is key range s of kv head h for
// row block blk, p = (h splits + s) nrb + blk; a CTA has every gridDim.x-th.
struct PrefixWalk {
  const SharedParams* p;
  int splits, tiles, extra;  // ranges of a segment: `tiles` tiles, the first `extra` of them one more
  int key_lo;                // first key of tile 0
  int slot, t, t1;           // piece, tile, end of the piece's tiles
  int h, blk;
  bool first;                // first tile of the piece
  __device__ __forceinline__ void begin(int piece) {
    slot = piece;
    const int hs = slot / p->s.nrb;
    blk = slot - hs * p->s.nrb;
    h = hs / splits;
    const int s = hs - h * splits;
    t = s * tiles + min(s, extra);
    t1 = t + tiles + (s < extra ? 1 : 0);
    first = true;
  }
  __device__ __forceinline__ int key0() const { return key_lo + T * t; }
  __device__ __forceinline__ bool last() const { return t == t1 - 1; }
  __device__ __forceinline__ void next() {
    first = false;
    if (++t == t1) begin(slot + gridDim.x);  // past the last piece: not used
  }
};

// A place in a CTA's run of own units: request, kv head, row block, tile.
struct OwnWalk {
  const SharedParams* p;
  int left;        // units from here to the end of the run
  int b, h, blk, seg, slot;
  int t, nt, n;    // tile of the segment, its tiles, own length
  bool first;      // first tile of this CTA's visit of the segment
  __device__ __forceinline__ void set_request() {
    n = min(p->own_len[b], p->g.own_rows);
    nt = own_tiles(p->g, n);
  }
  // unit r of request b0's segments
  __device__ __forceinline__ void begin(int b0, int r, int units) {
    b = b0;
    set_request();
    const int in = r / nt;
    t = r - in * nt;
    h = in / p->s.nomb;
    blk = in - h * p->s.nomb;
    slot = blockIdx.x + b * p->g.Hkv * p->s.nomb + in;
    left = units;
    first = true;
  }
  __device__ __forceinline__ int key0() const { return n - T * (nt - t); }
  __device__ __forceinline__ bool last() const { return left == 1 || t == nt - 1; }
  __device__ __forceinline__ void next() {
    first = false;
    ++t;
    if (--left == 0 || t < nt) return;
    first = true;
    t = 0;
    ++slot;
    if (++blk < p->s.nomb) return;
    blk = 0;
    if (++h < p->g.Hkv) return;
    h = 0;
    do {  // the next request with keys (there is one: units are left)
      ++b;
      set_request();
      slot += nt == 0 ? p->g.Hkv * p->s.nomb : 0;
    } while (nt == 0);
  }
};

// Shared memory of one phase: N query rows a block (own caches: 16).
template <int D, int N, bool OWN>
struct ShCfg {
  static constexpr int NCH = D / 64;             // 64-column chunks of a row
  static constexpr int CPS = NCH < 2 ? NCH : 2;  // chunks per ring slot
  static constexpr int SPT = NCH / CPS;          // slots per tile and tensor
  static constexpr int NDC = (D + 127) / 128;    // 128-column blocks of O^T
  static constexpr int NG = N > 16 ? 32 : 16;    // rows of a softmax warpgroup
  static constexpr int GROUPS = N / NG;
  static constexpr int SLOT = CPS * T * 128;
  static constexpr int QB = N * D * 2;           // one block of queries
  static constexpr int QD = OWN ? 2 : 1;         // blocks buffered (own segments are short)
  static constexpr int PB = N * T * 2;           // P^T
  // per warpgroup: [2][4][NG] exchanged maxima / sums, thresholds, references,
  // rescale factors, row ranges, bounds and tags
  static constexpr int SMALL = 2 * 4 * NG * 4 + 3 * NG * 4 + NG * 8 + 64;
  // at head dim 64 the second product's 128 rows read one chunk past a slot
  // (rows 64-127 of O^T, never used): the last slot's must stay in bounds
  static constexpr int TAIL = D == 64 ? T * 128 : 0;
  static constexpr int FIXED = QB * QD + PB + GROUPS * SMALL + TAIL;
  static constexpr int FIT = (kSmemMax - 1024 - 1024 - FIXED) / SLOT;
  // own caches stream from HBM on every SM: 128 KB in flight on each saturate
  // it, and more only lengthen the queues (4 slots of 32 KB against 6: 54.4 and
  // 55.8 us at 32 caches of up to 1,024 keys, D = 256; 3 slots: 56.0, and at
  // D = 512, where a tile has 8, 140 us against 118)
  static constexpr int MOST = OWN && CPS == 2 ? 4 : 8;
  static constexpr int NSLOT = FIT > MOST ? MOST : FIT;
  static constexpr int OFF_Q = NSLOT * SLOT;
  static constexpr int OFF_P = OFF_Q + QD * QB;
  static constexpr int OFF_SMALL = OFF_P + PB;
  static constexpr int BYTES = OFF_SMALL + GROUPS * SMALL + TAIL;
  // within a warpgroup's small arrays
  static constexpr int RED = 0, THR = 2 * 4 * NG * 4, USE = THR + NG * 4, ALPHA = USE + NG * 4, RNG = ALPHA + NG * 4,
                       BND = RNG + NG * 8;
  static constexpr uint32_t S_COL = 0, O_COL = 2 * N;  // TMEM columns
  static constexpr uint32_t COLS = O_COL + NDC * N;
  static_assert(NSLOT >= 2 && NSLOT <= 8, "ring slots (the barriers hold 8)");
  static_assert(COLS <= 512, "TMEM columns");
  static_assert(GROUPS <= 4, "softmax warpgroups");
};
template <int D, int NP>
struct ShKernel {
  using A = ShCfg<D, NP, false>;
  using B = ShCfg<D, kOwnRows, true>;
  static constexpr int THREADS = 64 + 128 * A::GROUPS;
  static constexpr int BODY = (A::BYTES > B::BYTES ? A::BYTES : B::BYTES);
  static constexpr int OFF_BAR = (BODY + 15) / 16 * 16;  // barriers of the two phases, 384 bytes each
  static constexpr size_t SMEM = (size_t)OFF_BAR + 768 + 1024;
  static constexpr uint32_t COLS = A::COLS > B::COLS ? A::COLS : B::COLS;
  static constexpr uint32_t TCOLS = COLS <= 128 ? 128 : (COLS <= 256 ? 256 : 512);
  static_assert(SMEM + 512 <= (size_t)kSmemMax, "shared memory");
};

// Column reduction over the warp's 32 lanes by halving: each step keeps one
// half of the columns and hands the other half over, so N columns take about
// N shuffles (5 N for a butterfly a column).  N = 32: lane l ends with column
// l in v[0]; N = 16: lanes 2 c, 2 c + 1 with column c.
template <int N, bool MAX>
__device__ __forceinline__ void column_reduce(float (&v)[N], int lane) {
  auto op = [](float a, float b) { return MAX ? fmaxf(a, b) : a + b; };
  int o = 16;
#pragma unroll
  for (int h = N / 2; h >= 1; h >>= 1, o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < h; ++i) {
      const float give = up ? v[i] : v[i + h], keep = up ? v[i + h] : v[i];
      v[i] = op(keep, __shfl_xor_sync(0xffffffffu, give, o));
    }
  }
  if (N == 16) v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], 1));
}
template <int N>
__device__ __forceinline__ void column_post(const float (&v)[N], float* dst, int lane) {
  if (N == 32) dst[lane] = v[0];
  else if ((lane & 1) == 0) dst[lane >> 1] = v[0];
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Waits for a phase as mbar_wait does, in a third of its code: the roles wait
// in some twenty places, and the code that a CTA runs once is fetched at the
// memory's latency (an unrolled 200 KB version of this kernel spent most of a
// short call on instruction fetches).
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint32_t t0 = (uint32_t)clock();
  do {
    if (mbar_try_wait(bar, parity)) return true;
  } while (!*abort && (uint32_t)clock() - t0 < 4000000000u);  // ~2 s, within the counter's 32 bits
  *abort = 1;
  return false;
}

// A phase's barriers (its own, so that none has to be set up twice).
struct Bars {
  uint64_t* b;
  __device__ __forceinline__ uint64_t* slot_full(int i) const { return b + i; }        // [8]
  __device__ __forceinline__ uint64_t* slot_empty(int i) const { return b + 8 + i; }   // [8]
  __device__ __forceinline__ uint64_t* q_full(int i) const { return b + 16 + i; }      // [2] a visit's queries
  __device__ __forceinline__ uint64_t* q_empty(int i) const { return b + 18 + i; }     // [2]
  __device__ __forceinline__ uint64_t* s_full(int i) const { return b + 20 + i; }      // [2] S^T(n) in TMEM
  __device__ __forceinline__ uint64_t* p_full() const { return b + 22; }  // P^T(n) written (and O^T rescaled)
  __device__ __forceinline__ uint64_t* o_done() const { return b + 23; }  // PV(n) finished
  __device__ __forceinline__ uint64_t* drain() const { return b + 24; }
  __device__ __forceinline__ uint64_t* xch(int i) const { return b + 25 + i; }  // [4] a softmax warpgroup's exchanges
  static constexpr int kCount = 29;
  // arrivals that complete a phase of barrier i
  static __device__ __forceinline__ int arrivals(int i, int groups) {
    return i == 22 ? 4 * groups : (i >= 25 ? 4 : 1);
  }
};

// What a softmax warpgroup works with.
struct SoftCtx {
  unsigned char* base;
  unsigned char* small;  // this warpgroup's small arrays
  Bars bar;
  volatile int* abort;
  uint32_t tmem;
  int group;
  int n;   // tiles done in this phase
  int xc;  // exchanges done
};

// Every softmax warp of the group arrives and waits (bounded); what was
// written to shared memory before is visible after.
__device__ __forceinline__ bool exchange(SoftCtx& c) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(c.bar.xch(c.group));
  const bool ok = wait(c.bar.xch(c.group), c.xc & 1, c.abort);
  ++c.xc;
  return __all_sync(0xffffffffu, ok);
}

// One visit of a segment: its tiles' softmax, then the partial result.  The
// rows' reference maxima live in shared memory; a tile only exchanges whether
// any score outgrew its row's threshold, which after a visit's first tile is
// rare (it also happens when a window first lets a row see a key).
template <int D, int N, bool OWN, typename Walk>
__device__ bool softmax_visit(const SharedParams& p, Walk& w, SoftCtx& c) {
  using C = ShCfg<D, N, OWN>;
  constexpr int NDC = C::NDC, NG = C::NG;
  const SharedGeom& g = p.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q4 = warp & 3, t = 32 * q4 + lane;
  const uint32_t lane_off = (uint32_t)(32 * q4) << 16, col0 = (uint32_t)(NG * c.group);
  const float sl2 = g.scale * kLog2e;
  float* red = reinterpret_cast<float*>(c.small + C::RED);
  float* thr = reinterpret_cast<float*>(c.small + C::THR);
  float* use = reinterpret_cast<float*>(c.small + C::USE);
  float* alp = reinterpret_cast<float*>(c.small + C::ALPHA);
  int2* rng = reinterpret_cast<int2*>(c.small + C::RNG);
  int* bnd = reinterpret_cast<int*>(c.small + C::BND);
  volatile int* grow_tag = bnd + 8;   // [2] tile (plus one) at which some score outgrew its threshold
  volatile int* scale_tag = bnd + 10;  // [1] tile (plus one) at which some row with earlier keys did
  const int blk = w.blk, slot = w.slot;

  // visible keys of row t (own cache: own indices), and bounds over all rows
  {
    int lo = 0, hi = INT32_MAX;  // rows that are no query mask nothing: their columns are never read
    bool row = false;
    if (t < NG) {
      const int r = NG * c.group + t;  // row of the block
      if constexpr (OWN) {
        const int m = blk * kOwnRows + r;
        row = m < g.M;
        if (row) {
          hi = w.n - g.Lq + m % g.Lq;
          lo = g.W > 0 ? max(0, hi - g.W + 1) : 0;
        }
      } else {
        const int b = blk / p.s.nmb * p.s.nb + r / p.s.mb, m = blk % p.s.nmb * N + r % p.s.mb;
        const int len = (r < p.s.prow && b < g.B && m < g.M) ? p.own_len[b] : -1;
        row = len >= 0;
        if (row) {
          const int a = g.P + min(len, g.own_rows) - g.Lq + m % g.Lq;
          hi = min(g.P - 1, a);
          lo = g.W > 0 ? max(0, a - g.W + 1) : 0;
        }
      }
      rng[t] = make_int2(lo, hi);
      thr[t] = -INFINITY;
    }
    const int lo_w = __reduce_max_sync(0xffffffffu, row ? lo : 0);
    const int hi_w = __reduce_min_sync(0xffffffffu, row ? hi : INT32_MAX);
    if (lane == 0) {
      bnd[q4 * 2] = lo_w;
      bnd[q4 * 2 + 1] = hi_w;
    }
  }
  if (!exchange(c)) return false;
  const int lo_all = max(max(bnd[0], bnd[2]), max(bnd[4], bnd[6]));
  const int hi_all = min(min(bnd[1], bnd[3]), min(bnd[5], bnd[7]));

  float l_part[NG], m_row = -INFINITY;  // thread t < NG holds row t's reference
#pragma unroll
  for (int q = 0; q < NG; ++q) l_part[q] = 0.f;

  bool more = true;
#pragma unroll 1
  while (more) {
    const int n = c.n, key0 = w.key0();
    const bool first = w.first;
    more = !w.last();
    if (!__all_sync(0xffffffffu, wait(c.bar.s_full(n & 1), (n >> 1) & 1, c.abort))) return false;
    tc_fence_after();
    uint32_t sr[NG];
    if constexpr (NG == 16) tmem_ld16(c.tmem + lane_off + C::S_COL + N * (n & 1) + col0, sr);
    else tmem_ld32(c.tmem + lane_off + C::S_COL + N * (n & 1) + col0, sr);
    tmem_wait_ld();
    float x[NG];
#pragma unroll
    for (int q = 0; q < NG; ++q) x[q] = __uint_as_float(sr[q]) * sl2;
    if (!(key0 >= lo_all && key0 + T - 1 <= hi_all)) {
      const int key = key0 + t;
#pragma unroll
      for (int q = 0; q < NG; ++q) {
        const int2 r = rng[q];
        if (key < r.x || key > r.y) x[q] = -INFINITY;
      }
    }
    bool grow = first, scale = false;
    if (!first) {
      bool over = false;
#pragma unroll
      for (int q = 0; q < NG; q += 4) {
        const float4 v = *reinterpret_cast<const float4*>(thr + q);
        over |= x[q] > v.x || x[q + 1] > v.y || x[q + 2] > v.z || x[q + 3] > v.w;
      }
      if (__any_sync(0xffffffffu, over) && lane == 0) grow_tag[n & 1] = n + 1;
      if (!exchange(c)) return false;
      grow = grow_tag[n & 1] == n + 1;
    }
    if (grow) {
      float* rb = red + (c.xc & 1) * 4 * NG;
      {
        float mx[NG];
#pragma unroll
        for (int q = 0; q < NG; ++q) mx[q] = x[q];
        column_reduce<NG, true>(mx, lane);
        column_post<NG>(mx, rb + q4 * NG, lane);
      }
      if (!exchange(c)) return false;
      if (t < NG) {
        const float tm = fmaxf(fmaxf(rb[t], rb[NG + t]), fmaxf(rb[2 * NG + t], rb[3 * NG + t]));
        float a = 1.f;
        if (tm > (m_row == -INFINITY ? m_row : m_row + kGrowLog2)) {
          if (m_row != -INFINITY) {
            a = fast_exp2(m_row - tm);
            *scale_tag = n + 1;
          }
          m_row = tm;
          use[t] = tm;
          thr[t] = tm + kGrowLog2;
        } else if (first) {
          use[t] = 0.f;  // no visible key yet
        }
        alp[t] = a;
      }
      if (!exchange(c)) return false;
      scale = *scale_tag == n + 1;
      if (scale) {
#pragma unroll
        for (int q = 0; q < NG; q += 4) {
          const float4 v = *reinterpret_cast<const float4*>(alp + q);
          l_part[q] *= v.x;
          l_part[q + 1] *= v.y;
          l_part[q + 2] *= v.z;
          l_part[q + 3] *= v.w;
        }
      }
    }
    // P = 2^(score - reference), two rows a word, and the row sums
    uint32_t pk[NG / 2];
#pragma unroll
    for (int q = 0; q < NG; q += 4) {
      const float4 v = *reinterpret_cast<const float4*>(use + q);
      const float e0 = fast_exp2(x[q] - v.x), e1 = fast_exp2(x[q + 1] - v.y);
      const float e2 = fast_exp2(x[q + 2] - v.z), e3 = fast_exp2(x[q + 3] - v.w);
      l_part[q] += e0;
      l_part[q + 1] += e1;
      l_part[q + 2] += e2;
      l_part[q + 3] += e3;
      pk[q / 2] = pack_bf16(e0, e1);
      pk[q / 2 + 1] = pack_bf16(e2, e3);
    }
    // PV(n - 1) has finished with P^T's buffer, and with O^T before it is rescaled
    if (n > 0 && !__all_sync(0xffffffffu, wait(c.bar.o_done(), (n - 1) & 1, c.abort))) return false;
    if (scale) {  // uniform over the warpgroup
      tc_fence_after();
#pragma unroll 1
      for (int i = 0; i < NDC * (NG / 16); ++i) {
        const int q0 = NG == 16 ? 0 : 16 * (i & 1);
        const uint32_t o_at = c.tmem + lane_off + C::O_COL + N * (NG == 16 ? i : i >> 1) + col0 + q0;
        uint32_t ov[16];
        tmem_ld16(o_at, ov);
        tmem_wait_ld();
#pragma unroll
        for (int q = 0; q < 16; ++q) ov[q] = __float_as_uint(__uint_as_float(ov[q]) * alp[q0 + q]);
        tmem_st16(o_at, ov);
      }
      tmem_wait_st();
    }
    unsigned char* pb = c.base + C::OFF_P;
    if constexpr (NG == 16) {
      // K-major B operand: row q, key t -> chunk t / 64, 128-byte swizzle
      pb += (t >> 6) * kOwnRows * 128 + (t & 7) * 2;
      const int kc = (t & 63) >> 3;
#pragma unroll
      for (int q = 0; q < 16; ++q)
        *reinterpret_cast<uint16_t*>(pb + q * 128 + ((kc ^ (q & 7)) << 4)) = (uint16_t)(pk[q / 2] >> (16 * (q & 1)));
    } else {
      // MN-major B operand: a key's 64 rows (two groups') are one 128-byte swizzled line
      pb += (c.group >> 1) * T * 128 + t * 128;
      const int u0 = 4 * (c.group & 1);
#pragma unroll
      for (int u = 0; u < 4; ++u)
        *reinterpret_cast<uint4*>(pb + (((u0 + u) ^ (t & 7)) << 4)) =
            make_uint4(pk[4 * u], pk[4 * u + 1], pk[4 * u + 2], pk[4 * u + 3]);
    }
    fence_proxy_async_smem();  // generic writes -> the tensor core's reads
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(c.bar.p_full());
    ++c.n;
    w.next();
  }

  // the visit's partial: row sums over the 128 threads, then O^T
  float* rb = red + (c.xc & 1) * 4 * NG;
  column_reduce<NG, false>(l_part, lane);
  column_post<NG>(l_part, rb + q4 * NG, lane);
  if (!exchange(c)) return false;
  if (!__all_sync(0xffffffffu, wait(c.bar.o_done(), (c.n - 1) & 1, c.abort))) return false;
  tc_fence_after();
  const int stride = OWN ? p.s.orow : p.s.prow;  // rows of a slot
  int rows;                                      // of which this segment has, and this group from row NG * group on
  if (OWN) rows = min(kOwnRows, g.M - blk * kOwnRows);
  else if (p.s.nmb > 1) rows = min(N, g.M - blk % p.s.nmb * N);
  else rows = min(p.s.nb, g.B - blk * p.s.nb) * g.M;
  rows -= NG * c.group;
  const size_t at = (size_t)slot * stride + NG * c.group;
  float* out = (OWN ? p.po_o : p.pp_o) + at * D;
  float* ml = (OWN ? p.po_ml : p.pp_ml) + at * 2;
  if (t < min(rows, NG))
    *reinterpret_cast<float2*>(ml + 2 * t) =
        make_float2(m_row, (rb[t] + rb[NG + t]) + (rb[2 * NG + t] + rb[3 * NG + t]));
#pragma unroll 1
  for (int h = 0; h < NDC; ++h) {
    float* dst = out + 128 * h + t;
#pragma unroll 1
    for (int q0 = 0; q0 < min(rows, NG); q0 += 16) {
      uint32_t ov[16];
      tmem_ld16(c.tmem + lane_off + C::O_COL + N * h + col0 + q0, ov);  // warp-collective
      tmem_wait_ld();
      if (128 * h + t < D) {
#pragma unroll
        for (int q = 0; q < 16; ++q)
          if (q0 + q < rows) dst[(q0 + q) * D] = __uint_as_float(ov[q]);
      }
    }
  }
  tc_fence_before();  // ordered before the next visit's first PV by its P arrival
  return true;
}

// One phase of a CTA's work: `total` tiles from walk `w0` on, all warp roles.
template <int D, int N, bool OWN, typename Walk>
__device__ void run_phase(const SharedParams& p, unsigned char* base, uint64_t* bar_mem, volatile int* abort_flag,
                          uint32_t tmem, const CUtensorMap* tmQ, const CUtensorMap* tmK, const CUtensorMap* tmV,
                          const Walk& w0, int total) {
  using C = ShCfg<D, N, OWN>;
  constexpr int NCH = C::NCH, CPS = C::CPS, SPT = C::SPT, NSLOT = C::NSLOT, QD = C::QD;
  const SharedGeom& g = p.g;
  const Bars bar{bar_mem};
  const int warp = threadIdx.x / 32;
  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (elect_one()) {
      Walk wk = w0, wv = w0;
      int issued = 0, nq = 0;
      auto load_tile = [&](Walk& w, const CUtensorMap* m) -> bool {
        const int key0 = w.key0();
        int head = w.h;
        if constexpr (OWN) head += w.b * g.Hkv;
#pragma unroll 1
        for (int sp = 0; sp < SPT; ++sp, ++issued) {
          const int s = issued % NSLOT;
          if (issued >= NSLOT && !wait(bar.slot_empty(s), ((issued / NSLOT) & 1) ^ 1, abort_flag)) return false;
          mbar_arrive_expect_tx(bar.slot_full(s), C::SLOT);
          tma_load_4d(base + s * C::SLOT, m, bar.slot_full(s), 0, key0, sp * CPS, head);
        }
        w.next();
        return true;
      };
      auto load_k = [&]() -> bool {
        if (wk.first) {
          const int s = nq % QD;
          if (nq >= QD && !wait(bar.q_empty(s), ((nq / QD) & 1) ^ 1, abort_flag)) return false;
          unsigned char* q = base + C::OFF_Q + s * C::QB;
          if constexpr (OWN) {
            mbar_arrive_expect_tx(bar.q_full(s), C::QB);
            tma_load_4d(q, tmQ, bar.q_full(s), 0, wk.blk * kOwnRows, 0, wk.b * g.Hkv + wk.h);
          } else {
            mbar_arrive_expect_tx(bar.q_full(s), NCH * p.s.prow * 128);
#pragma unroll 1
            for (int c = 0; c < NCH; ++c)
              tma_load_5d(q + c * N * 128, tmQ, bar.q_full(s), 0, wk.blk % p.s.nmb * N, c, wk.h,
                          wk.blk / p.s.nmb * p.s.nb);
          }
          ++nq;
        }
        return load_tile(wk, tmK);
      };
      // slots in MMA order: K(0), K(1), then per tile n: V(n), K(n + 2)
      bool ok = true;
#pragma unroll 1
      for (int n = -2; ok && n < total; ++n) ok = (n < 0 || load_tile(wv, tmV)) && (n + 2 >= total || load_k());
      if (*abort_flag) {  // unwinding: the loads in flight land before shared memory is released
        drain_ring(bar.q_full(0), QD, nq);
        drain_ring(bar.slot_full(0), NSLOT, issued);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (elect_one()) {
      const uint32_t idS = idesc_f16(T, N, 1, 1, 0, 0);                // K x Q^T, both K-major
      const uint32_t idPV = idesc_f16(T, N, 1, 1, 1, N > 16 ? 1 : 0);  // V^T (MN-major) x P^T
      Walk ws = w0, wv = w0;
      int used = 0, nq = 0;
      auto issue_s = [&](int n) -> bool {  // S^T(n) into buffer n & 1
        const int qs = nq % QD;
        if (ws.first && !wait(bar.q_full(qs), (nq / QD) & 1, abort_flag)) return false;
        uint64_t qd = smem_desc_sw128(smem_u32(base + C::OFF_Q + qs * C::QB), 16, 1024);
#pragma unroll 1
        for (int sp = 0; sp < SPT; ++sp, ++used) {
          const int s = used % NSLOT;
          if (!wait(bar.slot_full(s), (used / NSLOT) & 1, abort_flag)) return false;
          tc_fence_after();
          uint64_t kd = smem_desc_sw128(smem_u32(base + s * C::SLOT), 16, 1024);
#pragma unroll 1
          for (int cc = 0; cc < CPS; ++cc) {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              mma_ss(tmem + C::S_COL + N * (n & 1), desc_add(kd, ks * 32), desc_add(qd, ks * 32), idS,
                     (sp | cc | ks) ? 1u : 0u);
            kd = desc_add(kd, T * 128);
            qd = desc_add(qd, N * 128);
          }
          mma_commit(bar.slot_empty(s));
        }
        mma_commit(bar.s_full(n & 1));
        if (ws.last()) {  // the visit's queries are read
          mma_commit(bar.q_empty(qs));
          ++nq;
        }
        ws.next();
        return true;
      };
      const uint64_t pd = smem_desc_sw128(smem_u32(base + C::OFF_P), N > 16 ? T * 128 : 16, 1024);
      bool ok = true;
#pragma unroll 1
      for (int n = -2; ok && n < total; ++n) {
        if (n >= 0) {
          if (!wait(bar.p_full(), n & 1, abort_flag)) break;
          tc_fence_after();
          const uint32_t acc = wv.first ? 0u : 1u;
          // O^T block h (head-dim columns [128 h, 128 h + 128)) += V^T . P^T: one slot a block
#pragma unroll 1
          for (int h = 0; h < SPT; ++h, ++used) {
            const int s = used % NSLOT;
            if (!wait(bar.slot_full(s), (used / NSLOT) & 1, abort_flag)) { ok = false; break; }
            tc_fence_after();
            const uint64_t vd = smem_desc_sw128(smem_u32(base + s * C::SLOT), T * 128, 1024);  // MN-major
#pragma unroll
            for (int ks = 0; ks < T / 16; ++ks)
              mma_ss(tmem + C::O_COL + N * h, desc_add(vd, ks * 2048),
                     N > 16 ? desc_add(pd, ks * 2048) : desc_add(pd, (ks >> 2) * kOwnRows * 128 + (ks & 3) * 32),
                     idPV, (acc || ks > 0) ? 1u : 0u);
            mma_commit(bar.slot_empty(s));
          }
          if (!ok) break;
          mma_commit(bar.o_done());
          wv.next();
        }
        if (n + 2 < total) ok = issue_s(n + 2);  // after PV(n): S buffer n & 1 is free
      }
      mma_commit(bar.drain());
      mbar_wait_drain(bar.drain(), 0);
    }
  } else if ((warp - 2) / 4 < C::GROUPS) {
    // ------------------------------------------------------------ softmax
    const int group = (warp - 2) / 4;
    SoftCtx c{base, base + C::OFF_SMALL + group * C::SMALL, bar, abort_flag, tmem, group, 0, 0};
    Walk w = w0;
    bool ok = true;
#pragma unroll 1
    while (ok && c.n < total) ok = softmax_visit<D, N, OWN>(p, w, c);
  }
  __syncwarp();
}

template <int D, int NP>
__global__ void __launch_bounds__(ShKernel<D, NP>::THREADS, 1)
    shared_kernel(const __grid_constant__ CUtensorMap tmQP, const __grid_constant__ CUtensorMap tmQO,
                  const __grid_constant__ CUtensorMap tmKP, const __grid_constant__ CUtensorMap tmVP,
                  const __grid_constant__ CUtensorMap tmKO, const __grid_constant__ CUtensorMap tmVO,
                  const __grid_constant__ SharedParams p) {
  using K = ShKernel<D, NP>;
  using A = typename K::A;
  constexpr int THR = K::THREADS, NW = THR / 32;
  extern __shared__ unsigned char smem_raw[];
  __shared__ int scan_sum[NW], scan_min[NW], start_b, start_r;
  __shared__ unsigned scan_best[NW];
  unsigned char* base = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(base + K::OFF_BAR);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 32);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint64_t* bars2 = bars + 48;

  const SharedGeom& g = p.g;
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    start_b = -1;
    *abort_flag = 0;
    prefetch_tmap(&tmKP);
    prefetch_tmap(&tmKO);
  }
  if (threadIdx.x < 64 && lane < Bars::kCount) {
    mbar_init((warp ? bars2 : bars) + lane, Bars::arrivals(lane, warp ? 1 : A::GROUPS));
    fence_mbar_init();
  }
  // rows of the prefix query block that no box fills stay zero
#pragma unroll 1
  for (int i = threadIdx.x; i < A::QB / 16; i += THR) reinterpret_cast<uint4*>(base + A::OFF_Q)[i] = make_uint4(0, 0, 0, 0);
  if (threadIdx.x < 4 * A::GROUPS)  // tags of the prefix phase
    reinterpret_cast<int*>(base + A::OFF_SMALL + (threadIdx.x >> 2) * A::SMALL + A::BND)[8 + (threadIdx.x & 3)] = 0;
  fence_proxy_async_smem();
  grid_dependency_wait();
  // Tensor memory is taken after the predecessor's end and before a dependent
  // may be placed: a grid that held columns while it waits for another that has
  // yet to allocate its own, on the same SM, would wait for ever.
  if (warp == 1) {
    tmem_alloc(tmem_slot, K::TCOLS);
    tmem_relinquish();
  }
  // ---- the lengths: own tiles in all, the shortest live request
  {
    int sum = 0, mn = INT32_MAX;
#pragma unroll 1
    for (int b = threadIdx.x; b < g.B; b += THR) {
      const int len = p.own_len[b];
      sum += own_tiles(g, len);
      if (len >= 0) mn = min(mn, min(len, g.own_rows));
    }
    sum = __reduce_add_sync(0xffffffffu, sum);
    mn = __reduce_min_sync(0xffffffffu, mn);
    if (lane == 0) {
      scan_sum[warp] = sum;
      scan_min[warp] = mn;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_launch_dependents();  // the merge waits for this grid's end
  const uint32_t tmem = *tmem_slot;
  int tiles = 0, mn = INT32_MAX;
#pragma unroll
  for (int i = 0; i < NW; ++i) {
    tiles += scan_sum[i];
    mn = min(mn, scan_min[i]);
  }

  // ---- the split.  Prefix keys that some row sees start at key_lo (there are
  // none without a live request); tp tiles of nseg segments, in ns ranges each
  constexpr int ctas = kSMs;
  const int cta = blockIdx.x;
  const int key_lo = mn == INT32_MAX ? g.P : (g.W > 0 ? min(g.P, max(0, g.P + mn - g.Lq - g.W + 1)) : 0);
  const int tp = (g.P - key_lo + T - 1) / T;
  const int nseg = tp > 0 ? g.Hkv * p.s.nrb : 0, hn = g.Hkv * p.s.nomb, own_units = tiles * hn;
  // ns: the one that makes the longest CTA's units fewest, a piece counting one
  // unit more than its tiles (its queries' load and its partial's store)
  const int most = nseg ? min(tp, max(1, kPieces / nseg)) : 0;
  {
    unsigned mine = ~0u;
#pragma unroll 1
    for (int i = 1 + threadIdx.x; i <= most; i += THR) {
      const int np = nseg * i, k = (np + ctas - 1) / ctas;
      const int all = (nseg * tp + np + own_units + ctas - 1) / ctas;
      mine = min(mine, (unsigned)min(max(k * ((tp + i - 1) / i + 1), all), 0x3fffff) << 9 | i);
    }
    mine = __reduce_min_sync(0xffffffffu, mine);
    if (lane == 0) scan_best[warp] = mine;
  }
  __syncthreads();
  unsigned best = ~0u;
#pragma unroll
  for (int i = 0; i < NW; ++i) best = min(best, scan_best[i]);
  const int ns = nseg ? best & 511 : 1, pieces = nseg * ns;
  // own runs fill the CTAs up to the same number of units: the first `rich`
  // CTAs have `rounds` pieces, the others one less
  const int rounds = (pieces + ctas - 1) / ctas, rich = pieces - (rounds > 0 ? rounds - 1 : 0) * ctas;
  const int pl = pieces ? (tp + ns - 1) / ns + 1 : 0, even = (own_units + pieces * pl + ctas - 1) / ctas;
  const int qa = max(0, even - rounds * pl);  // own units of a rich CTA, and of another
  const int qb = qa > 0 || rich == ctas ? even - (rounds - 1) * pl : (own_units + ctas - rich - 1) / (ctas - rich);
  const OwnRuns runs{rich, qa, qb, own_units};
  const int o0 = runs.start(cta), o1 = runs.start(cta + 1);
  if (cta == 0 && threadIdx.x == 0) {  // for the merge
    *reinterpret_cast<int4*>(p.plan) = make_int4(tp, ns, rich, qa);
    *reinterpret_cast<int4*>(p.plan + 4) = make_int4(qb, own_units, 0, 0);
  }
  // the request that own unit o0 belongs to; CTA 0 also writes every request's
  // first tile for the merge
  if (o0 < o1 || cta == 0) {
    int before = 0;
#pragma unroll 1
    for (int c0 = 0; c0 < g.B; c0 += THR) {
      const int b = c0 + threadIdx.x;
      const int nt = b < g.B ? own_tiles(g, p.own_len[b]) : 0;
      int inc = nt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      __syncthreads();
      if (lane == 31) scan_sum[warp] = inc;
      __syncthreads();
      int off = before + inc - nt;
      for (int i = 0; i < NW; ++i) {
        if (i < warp) off += scan_sum[i];
        before += scan_sum[i];
      }
      if (cta == 0 && b < g.B) p.plan[kPlanOff + b] = off;
      if (nt > 0 && o0 >= off * hn && o0 < (off + nt) * hn) {
        start_b = b;
        start_r = o0 - off * hn;
      }
    }
    __syncthreads();
  }

  // ---- the prefix pieces, then the own run
  if (cta < pieces) {
    PrefixWalk w;
    w.p = &p;
    w.splits = ns;
    w.tiles = tp / ns;
    w.extra = tp - ns * w.tiles;
    w.key_lo = key_lo;
    int total = 0;
#pragma unroll 1
    for (int i = cta; i < pieces; i += ctas) {
      w.begin(i);
      total += w.t1 - w.t;
    }
    w.begin(cta);
    run_phase<D, NP, false>(p, base, bars, abort_flag, tmem, &tmQP, &tmKP, &tmVP, w, total);
  }
  if (o0 < o1) {
    if (cta < pieces) {  // the shared memory and the accumulators change hands
      fence_proxy_async_smem();  // the small arrays' generic accesses, before loads that land there
      tc_fence_before();
      __syncthreads();
      tc_fence_after();
    }
    if (threadIdx.x < 4)  // tags of this phase
      reinterpret_cast<int*>(base + K::B::OFF_SMALL + K::B::BND)[8 + threadIdx.x] = 0;
    __syncthreads();
    if (!*abort_flag) {
      OwnWalk w;
      w.p = &p;
      w.begin(start_b, start_r, o1 - o0);
      run_phase<D, kOwnRows, true>(p, base, bars2, abort_flag, tmem, &tmQO, &tmKO, &tmVO, w, o1 - o0);
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (*abort_flag && threadIdx.x == 0) atomicCAS(p.status, 0, kStatusTimeout);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, K::TCOLS);
  }
}

// Merge of one query row's partials: those of its prefix block's pieces, and
// of its own cache, one for each CTA that had a part of the segment (they are
// neighbours).  Rows without a key get o = 0 and lse = -inf (or the sink's
// logit); rows of an empty place of the batch are not written.
//
// A row's partials are a few KB spread over L2, so the memory's latency is what
// this takes: D / 4 threads read a partial, THREADS / (D / 4) partials are read
// at once, with AHEAD loads a thread under way before the weights are known,
// and every warp forms the weights by itself.  THREADS: 256 where that is at
// most two CTAs an SM, else 128 (a call's time with 256 and 128: 256 rows of
// some 40 partials, D = 128: 15.1 and 17.0 us; 1,024 rows of as many, D = 64:
// 19.2 and 16.3; 2,048 rows of 11, D = 512: 122 and 119).
template <int D, int THREADS>
__global__ void __launch_bounds__(THREADS) shared_merge_kernel(const __grid_constant__ SharedParams p) {
  constexpr int LANES = D / 4, GR = THREADS / LANES, AHEAD = 1024 / THREADS;
  __shared__ float4 part[GR][LANES];
  const SharedGeom& g = p.g;
  const SharedSplit& s = p.s;
  const int row = blockIdx.x;  // (b Hkv + kv head) M + m
  const int bkv = row / g.M, m = row - bkv * g.M, b = bkv / g.Hkv, h = bkv - b * g.Hkv;
  const int lane = threadIdx.x & 31, grp = threadIdx.x / LANES, d = threadIdx.x % LANES;
  grid_launch_dependents();
  // the main grid lets this one start once it has waited for what wrote the lengths
  const int len = __ldcg(p.own_len + b);
  const float* sink = p.sinks ? p.sinks + h * g.G + m / g.Lq : nullptr;
  const int nt = own_tiles(g, len), hn = g.Hkv * s.nomb, in = h * s.nomb + m / kOwnRows;
  const int rb = s.nmb > 1 ? b * s.nmb + m / s.np : b / s.nb;
  const int q = s.nmb > 1 ? m % s.np : b % s.nb * g.M + m;
  const size_t o_seg = (size_t)(b * hn + in) * s.orow + m % kOwnRows, p_step = (size_t)s.nrb * s.prow;
  grid_dependency_wait();
  if (len < 0) return;
  const int4 pl = *reinterpret_cast<const int4*>(p.plan), pr = *reinterpret_cast<const int4*>(p.plan + 4);
  const int off = p.plan[kPlanOff + b];
  // the row's partials: np of its prefix block, ns pieces, then those of the
  // CTAs whose own run meets its segment
  const int np = pl.x > 0 ? pl.y : 0;
  const OwnRuns runs{pl.z, pl.w, pr.x, pr.y};
  const int u0 = off * hn + in * nt, c0 = nt > 0 ? runs.owner(u0) : 0, n = np + (nt > 0 ? runs.owner(u0 + nt - 1) - c0 + 1 : 0);
  const size_t p_at = ((size_t)h * pl.y * s.nrb + rb) * s.prow + q, o_at = o_seg + (size_t)c0 * s.orow;
  auto row_of = [&](int i) {  // partial i: its row among the prefix's or the own partials
    return i < np ? p_at + i * p_step : o_at + (size_t)(i - np) * s.orow;
  };
  auto ml_of = [&](int i) { return *reinterpret_cast<const float2*>((i < np ? p.pp_ml : p.po_ml) + row_of(i) * 2); };
  auto o_of = [&](int i) { return *reinterpret_cast<const float4*>((i < np ? p.pp_o : p.po_o) + row_of(i) * D + 4 * d); };
  // all first loads are under way before any is used
  const float2 first = lane < n ? ml_of(lane) : make_float2(-INFINITY, 0.f);
  float4 v[AHEAD];
  float mi[AHEAD];
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) {
    const int j = grp + GR * i;
    if (j < n) {
      v[i] = o_of(j);
      mi[i] = ml_of(j).x;
    }
  }
  // a part without a visible key adds nothing (its l is 0; NaN scores leave no
  // maximum either, and a NaN l)
  float mx = first.x;
#pragma unroll 1
  for (int i = lane + 32; i < n; i += 32) mx = fmaxf(mx, ml_of(i).x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  auto weight = [&](float x) { return x == -INFINITY ? 0.f : exp2f(x - mx); };
  float l = first.x == -INFINITY ? first.y : weight(first.x) * first.y;
#pragma unroll 1
  for (int i = lane + 32; i < n; i += 32) {
    const float2 t = ml_of(i);
    l += t.x == -INFINITY ? t.y : weight(t.x) * t.y;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](float w, const float4& u) {
    acc.x = fmaf(w, u.x, acc.x);
    acc.y = fmaf(w, u.y, acc.y);
    acc.z = fmaf(w, u.z, acc.z);
    acc.w = fmaf(w, u.w, acc.w);
  };
#pragma unroll
  for (int i = 0; i < AHEAD; ++i)
    if (grp + GR * i < n) add(weight(mi[i]), v[i]);
#pragma unroll 4
  for (int j = grp + GR * AHEAD; j < n; j += GR) add(weight(ml_of(j).x), o_of(j));
  part[grp][d] = acc;
  __syncthreads();
  if (grp > 0) return;
#pragma unroll
  for (int i = 1; i < GR; ++i) add(1.f, part[i][d]);
  float inv, lse;
  if (mx == -INFINITY && l == 0.f) {
    inv = 0.f;
    lse = sink ? *sink : -INFINITY;
  } else {
    inv = 1.f / l;
    lse = (mx + log2f(l)) * kLn2;
    if (sink) inv = sink_finish(*sink, mx, l, &lse);
  }
  *reinterpret_cast<uint2*>(p.o + (size_t)row * D + 4 * d) =
      make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
  if (d == 0) p.lse[row] = lse;
}

struct SharedWs {
  size_t plan, pp_ml, pp_o, po_ml, po_o, total;
};
SharedWs shared_ws(const SharedGeom& g) {
  const SharedSplit s = shared_split(g);
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const long long nseg = (long long)g.Hkv * s.nrb;
  const size_t ps = (size_t)(nseg > kPieces ? nseg : kPieces) * s.prow, os = (size_t)(kSMs + (long long)g.B * g.Hkv * s.nomb) * s.orow;
  SharedWs w;
  w.plan = 0;
  w.pp_ml = w.plan + up(((size_t)g.B + kPlanOff) * 4);
  w.pp_o = w.pp_ml + (g.P > 0 ? up(ps * 8) : 0);
  w.po_ml = w.pp_o + (g.P > 0 ? up(ps * g.D * 4) : 0);
  w.po_o = w.po_ml + up(os * 8);
  w.total = w.po_o + up(os * g.D * 4);
  return w;
}

template <int D, int NP>
cudaError_t shared_d(const SharedGeom& g, const SharedArgs& a, void* ws, int* status, cudaStream_t st) {
  using K = ShKernel<D, NP>;
  constexpr int CPS = K::A::CPS;
  const SharedSplit s = shared_split(g);
  CUtensorMap tqp, tqo, tkp, tvp, tko, tvo;
  cudaError_t e;
  if ((e = make_tmap_rows_5d(&tqp, a.q, D, g.M, g.Hkv, g.B, s.mb, s.nb)) != cudaSuccess) return e;
  if ((e = make_tmap_f16_chunks(&tqo, a.q, D, g.M, g.B * g.Hkv, kOwnRows, D / 64)) != cudaSuccess) return e;
  if ((e = make_tmap_f16_chunks(&tko, a.ko, D, g.own_rows, g.B * g.Hkv, T, CPS)) != cudaSuccess) return e;
  if ((e = make_tmap_f16_chunks(&tvo, a.vo, D, g.own_rows, g.B * g.Hkv, T, CPS)) != cudaSuccess) return e;
  if (g.P > 0) {
    // rows at or beyond the prefix's length read as zero
    if ((e = make_tmap_f16_chunks(&tkp, a.kp, D, g.P, g.Hkv, T, CPS, g.prefix_rows)) != cudaSuccess) return e;
    if ((e = make_tmap_f16_chunks(&tvp, a.vp, D, g.P, g.Hkv, T, CPS, g.prefix_rows)) != cudaSuccess) return e;
  } else {
    tkp = tko;  // not used: the prefix has no tiles
    tvp = tvo;
  }
  const SharedWs w = shared_ws(g);
  unsigned char* wb = static_cast<unsigned char*>(ws);
  SharedParams p;
  p.g = g;
  p.s = s;
  p.own_len = a.own_len;
  p.sinks = a.sinks;
  p.o = a.o;
  p.lse = a.lse;
  p.plan = reinterpret_cast<int*>(wb + w.plan);
  p.pp_ml = reinterpret_cast<float*>(wb + w.pp_ml);
  p.pp_o = reinterpret_cast<float*>(wb + w.pp_o);
  p.po_ml = reinterpret_cast<float*>(wb + w.po_ml);
  p.po_o = reinterpret_cast<float*>(wb + w.po_o);
  p.status = status;
  auto kern = shared_kernel<D, NP>;
  if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)K::SMEM)) != cudaSuccess)
    return e;
  // both are programmatic dependents of what runs before them: the main grid's
  // set-up and the merge's placement fall into its predecessor's end
  if ((e = launch_dependent(kern, dim3(kSMs), dim3(K::THREADS), K::SMEM, st, tqp, tqo, tkp, tvp, tko, tvo, p)) !=
      cudaSuccess)
    return e;
  const unsigned rows = (unsigned)(g.B * g.Hkv * g.M);
  if (rows <= 2 * kSMs) return launch_dependent(shared_merge_kernel<D, 256>, dim3(rows), dim3(256), 0, st, p);
  return launch_dependent(shared_merge_kernel<D, 128>, dim3(rows), dim3(128), 0, st, p);
}

template <int D>
cudaError_t shared_np(const SharedGeom& g, const SharedArgs& a, void* ws, int* status, cudaStream_t st) {
  switch (shared_split(g).np) {
    case 16: return shared_d<D, 16>(g, a, ws, status, st);
    case 64: return shared_d<D, 64>(g, a, ws, status, st);
    default:
      if constexpr (D <= 256) return shared_d<D, 128>(g, a, ws, status, st);
      else return cudaErrorInvalidValue;
  }
}

}  // namespace

SharedSplit shared_split(const SharedGeom& g) {
  SharedSplit s;
  // (at D = 512 the accumulators of 128 rows would not fit beside the scores)
  const long long r = (long long)g.B * g.M;
  s.np = r <= 16 ? 16 : (r <= 64 || g.D == 512 ? 64 : 128);
  s.mb = g.M < s.np ? g.M : s.np;
  s.nmb = (g.M + s.np - 1) / s.np;
  s.nb = g.M <= s.np ? s.np / g.M : 1;
  if (s.nb > g.B) s.nb = g.B;
  s.prow = s.nb * s.mb;
  s.nrb = s.nmb > 1 ? g.B * s.nmb : (g.B + s.nb - 1) / s.nb;
  s.nomb = (g.M + kOwnRows - 1) / kOwnRows;
  s.orow = g.M < kOwnRows ? g.M : kOwnRows;
  return s;
}

bool shared_fits(const SharedGeom& g) {
  const SharedSplit s = shared_split(g);
  const double tp = (g.P + T - 1) / T, to = (g.own_rows + T - 1) / T;
  const double units = (double)g.Hkv * s.nrb * tp + (double)g.B * g.Hkv * s.nomb * to;
  return units + kPieces < 1.0e9 && (double)g.B * g.Hkv * g.M < 1.0e9 && (double)g.B * g.Hkv * s.nomb < 1.0e9;
}

size_t shared_workspace_bytes(const SharedGeom& g) { return shared_ws(g).total; }

cudaError_t launch_fwd_shared(const SharedGeom& g, const SharedArgs& a, void* ws, int* status, cudaStream_t st) {
  switch (g.D) {
    case 64: return shared_np<64>(g, a, ws, status, st);
    case 128: return shared_np<128>(g, a, ws, status, st);
    case 256: return shared_np<256>(g, a, ws, status, st);
    case 512: return shared_np<512>(g, a, ws, status, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace swa
