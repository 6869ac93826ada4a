// Attention of a generation step for a batch that shares a long prefix: every
// request's queries see the prefix's keys, kept once for all of them, and the
// keys of the request's own cache, whose length only the device knows.
//
// For request b with own length n, query row i (of Lq) sits at position
// a = P + n - Lq + i behind the P prefix keys and sees the keys j <= a of
// [prefix; own cache] with a - j < W (W = 0: all of them).  A softmax over two
// key sets splits exactly: each set (and each part of one) gives its reference
// m, its sum l of 2^(s - m) and its unnormalised O, and with M = max m
//   o = sum 2^(m - M) O / sum 2^(m - M) l,   lse = (M + log2 sum 2^(m - M) l) ln 2.
//
// Work.  The unit is one key tile (T = 128 keys) of one segment.  A segment is
// the product of one block of query rows with one kv head's prefix (up to N
// rows, packed from as many requests as fit, so the prefix is read once for
// all of them), or with one request's own cache (up to 16 rows: the G * Lq
// rows of a kv head).  One CTA per SM works first on pieces of the prefix,
// then on a run of the requests' own tiles, so that all CTAs take the same
// time however ragged the lengths are: every CTA sums the device-side lengths
// itself, no host sees them, and no counter has to be reset between calls.
// Pieces of one key range with all its row blocks are neighbouring CTAs' work
// at the same time, so a tile's second and later reads find it in L2 (64
// requests of 32 heads over 16,384 keys, D = 512: 139 MB from HBM and 127 us;
// with pieces that drift apart 1.2 GB and 208 us).  Each piece, and each CTA's
// share of an own segment, leaves one partial (m, l, O) in a slot of its own; a
// second kernel merges a row's partials.
//
// Bounds, of 64 requests of 32 heads (4 of them kv) over 16,384 prefix keys and
// up to 1,024 of their own, D = 512 (104 us): the prefix's tiles, 2.2 us each
// where L2 has them, are bound by shared memory (a tile's operands are 393 KB of
// MMA reads and 256 KB of TMA writes: 2.5 us if each byte took its turn at 128 a
// clock); the own caches by HBM (32 caches of up to 1,024 keys at D = 256: 6.0
// TB/s of a whole call).  At D <= 128 a prefix tile is bound by the softmax's
// latency (1.3 us for 64 rows, 1.8 for 128 at D = 64 and 2.0 at D = 128), and a
// short call by what comes before and behind: lengths 0.5 us, split 0.7, first
// tile 1.3, merge 1.8 (4 requests over 1,024 keys, D = 128: 7.9 us, of which 1.6
// are tiles).
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

#include <type_traits>

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
// A row's reference is 2^16 above the largest score of its first tile with a
// visible key, and only moves when a score outgrows it.  So P = 2^(score -
// reference) is never above 1, and O never larger than with the maximum itself
// as the reference: values of any size that the products' sum can hold are
// safe.  What lies below costs nothing down to 2^-110 of the largest weight
// (P, its sums and O are bf16 and fp32, whose precision is relative).
constexpr float kRoomLog2 = 16.0f;
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
  int prefix_pass;     // whether the prefix gives way in L2
  int most;            // ranges that a prefix segment is split into at most
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
    const int nrb = p->s.nrb, hs = nrb > 1 ? slot / nrb : slot;
    blk = slot - hs * nrb;
    // hs < 2^20 where there are splits (they make at most kPieces pieces), and a
    // quotient's distance from the next is 1 / (2 splits) at least
    h = splits > 1 ? (int)__fdividef(hs + 0.5f, (float)splits) : hs;
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
  __device__ __forceinline__ int skip() {  // over the rest of the visit; its tiles
    const int k = min(left, nt - t);
    t += k - 1;
    left -= k - 1;
    next();
    return k;
  }
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

// One phase's blocks of N query rows (own caches: 16).
template <int D, int N>
struct ShPhase {
  static constexpr int NG = N > 16 ? 32 : 16;  // rows of a softmax warpgroup
  static constexpr int QB = N * D * 2;         // a block of queries
  static constexpr int PB = N * T * 2;         // P^T
  // a softmax warpgroup's small arrays: [2][4][NG] exchanged maxima / sums, thresholds, references, rescale
  // factors, row ranges, bounds and tags
  static constexpr int RED = 0, THR = 2 * 4 * NG * 4, USE = THR + NG * 4, ALPHA = USE + NG * 4, RNG = ALPHA + NG * 4,
                       BND = RNG + NG * 8, SMALL = BND + 64;
};
// The kernel with prefix blocks of N rows.  Shared memory: one ring of slots for
// both phases, the prefix blocks' queries and P^T, and the own caches', which
// take over the same bytes where these are large enough.
template <int D, int N>
struct ShKernel {
  using A = ShPhase<D, N>;
  using B = ShPhase<D, kOwnRows>;
  static constexpr int NCH = D / 64;             // 64-column chunks of a row
  static constexpr int CPS = NCH < 2 ? NCH : 2;  // chunks per ring slot
  static constexpr int SPT = NCH / CPS;          // slots per tile and tensor
  static constexpr int NDC = (D + 127) / 128;    // 128-column blocks of O^T
  static constexpr int SLOT = CPS * T * 128;
  static constexpr int GROUPS = N / A::NG;       // softmax warpgroups of the prefix; own segments take turns in two
  // The split's weights, in about quarter microseconds of a full GPU (a tile whose
  // operands L2 has takes up to a third less): a prefix tile, an own tile, what a
  // piece adds to its tiles, what an own run adds
  static constexpr int WP = N == 128 ? (D == 256 ? 12 : D == 128 ? 10 : 9)
                                     : (D == 512 ? 11 : D == 256 ? (N == 64 ? 7 : 9) : (N == 64 ? 5 : 4));
  static constexpr int WO = D == 512 ? 11 : D == 256 ? (N == 128 ? 12 : 7) : D == 128 ? (N == 128 ? 9 : 4) : (N == 128 ? 5 : 4);
  static constexpr int VP = D == 512 ? 14 : 6, WV = 4;
  static constexpr int THREADS = 64 + 128 * (GROUPS > 2 ? GROUPS : 2);
  // few rows: at most 128 registers a thread, so that merge CTAs are placed
  // beside this one's while they run (with more rows it would spill)
  static constexpr int BOUND = N == 16 ? 512 : THREADS;
  static constexpr bool SHARE_Q = A::QB >= 2 * B::QB, SHARE_P = A::PB >= 2 * B::PB;
  // at head dim 64 the second product's 128 rows read one chunk past a slot
  // (rows 64-127 of O^T, never used): the last slot's must stay in bounds
  static constexpr int TAIL = D == 64 ? T * 128 : 0;
  static constexpr int FIXED = A::QB + A::PB + (SHARE_Q ? 0 : 2 * B::QB) + (SHARE_P ? 0 : 2 * B::PB) +
                               GROUPS * A::SMALL + 2 * B::SMALL;
  static constexpr int FIT = (kSmemMax - 1024 - 1024 - FIXED - TAIL) / SLOT;
  static constexpr int NSLOT = FIT > 8 ? 8 : FIT;
  // own caches stream from HBM on every SM: 128 KB in flight on each saturate
  // it, and more only lengthen the queues (4 slots of 32 KB against 6: 54.4 and
  // 55.8 us at 32 caches of up to 1,024 keys, D = 256; 3 slots: 56.0, and at
  // D = 512, where a tile has 8, 140 us against 118)
  static constexpr int OWN_AHEAD = CPS == 2 && NSLOT > 4 ? 4 : NSLOT;
  static constexpr int OFF_Q = NSLOT * SLOT, OFF_P = OFF_Q + A::QB, END_P = OFF_P + A::PB;
  static constexpr int OFF_QO = SHARE_Q ? OFF_Q : END_P;
  static constexpr int END_QO = SHARE_Q ? END_P : END_P + 2 * B::QB;
  static constexpr int OFF_PO = SHARE_P ? OFF_P : END_QO;
  static constexpr int OFF_SMALL = SHARE_P ? END_QO : END_QO + 2 * B::PB;
  static constexpr int OFF_SMALL_O = OFF_SMALL + GROUPS * A::SMALL;
  static constexpr int BODY = OFF_SMALL_O + 2 * B::SMALL;
  static constexpr int OFF_BAR = ((BODY > OFF_Q + TAIL ? BODY : OFF_Q + TAIL) + 15) / 16 * 16;
  static constexpr int OFF_ABORT = OFF_BAR + 48 * 8 + 8;  // behind the barriers and the TMEM address
  static constexpr size_t SMEM = (size_t)OFF_BAR + 512 + 1024;
  // TMEM columns: S^T twice and O^T of the prefix.  The own segments' O^T (one
  // for each warpgroup) and S^T lie where the prefix's scores were, which have
  // all been read before the first own product is issued, or behind.
  static constexpr uint32_t S_COL = 0, O_COL = 2 * N, A_END = O_COL + NDC * N;
  static constexpr bool O_IN_S = 2 * N >= 32 * NDC, S_IN_S = 2 * N >= 32 * NDC + 32;
  static constexpr uint32_t O_OWN = O_IN_S ? 0 : A_END, S_OWN = S_IN_S ? 32 * NDC : (O_IN_S ? A_END : A_END + 32 * NDC);
  static constexpr uint32_t COLS = S_IN_S ? A_END : S_OWN + 32;
  static constexpr uint32_t TCOLS = COLS <= 128 ? 128 : (COLS <= 256 ? 256 : 512);
  static_assert(NSLOT >= 2 && NSLOT <= 8, "ring slots (the barriers hold 8)");
  static_assert(COLS <= 512, "TMEM columns");
  static_assert(GROUPS <= 4, "softmax warpgroups");
  static_assert(SMEM + 512 <= (size_t)kSmemMax, "shared memory");
  static_assert(OFF_QO % 1024 == 0 && OFF_PO % 1024 == 0 && OFF_P % 1024 == 0, "swizzled tiles");
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

// Barriers.  The ring's are shared by both phases; each has its own for the
// rest, the own segments' one set a warpgroup.
struct Bars {
  uint64_t* b;
  __device__ __forceinline__ uint64_t* slot_full(int i) const { return b + i; }       // [8]
  __device__ __forceinline__ uint64_t* slot_empty(int i) const { return b + 8 + i; }  // [8]
  __device__ __forceinline__ uint64_t* drain() const { return b + 16; }
  template <bool OWN>
  __device__ __forceinline__ uint64_t* q_full(int i) const { return b + (OWN ? 27 : 17) + i; }  // a visit's queries (own: [2])
  template <bool OWN>
  __device__ __forceinline__ uint64_t* q_empty(int i) const { return b + (OWN ? 29 : 18) + i; }
  template <bool OWN>
  __device__ __forceinline__ uint64_t* s_full(int g) const { return b + (OWN ? 31 + 2 * g : 19); }  // [2] S^T in TMEM
  template <bool OWN>
  __device__ __forceinline__ uint64_t* p_full(int g) const { return b + (OWN ? 35 + g : 21); }  // P^T written (O^T rescaled)
  template <bool OWN>
  __device__ __forceinline__ uint64_t* o_done(int g) const { return b + (OWN ? 37 + g : 22); }  // PV finished
  template <bool OWN>
  __device__ __forceinline__ uint64_t* xch(int g) const { return b + (OWN ? 39 : 23) + g; }  // a warpgroup's exchanges
  static constexpr int kCount = 41;
  // arrivals that complete a phase of barrier i
  static __device__ __forceinline__ int arrivals(int i, int groups) {
    return i == 21 ? 4 * groups : ((i >= 23 && i < 27) || i == 35 || i == 36 || i >= 39 ? 4 : 1);
  }
};

// A softmax warpgroup's place in a phase.
template <int D, int NP, bool OWN>
struct SoftCtx {
  using K = ShKernel<D, NP>;
  using C = typename std::conditional<OWN, typename K::B, typename K::A>::type;
  unsigned char* base;
  uint32_t at;   // TMEM: this thread's lane
  int group;
  int n;         // the phase's tiles so far: S^T(n) is in buffer n & 1
  int k;         // of which this warpgroup has done k
  uint32_t sph;  // phases of s_full
  int xc;        // exchanges done
  __device__ __forceinline__ Bars bar() const { return Bars{reinterpret_cast<uint64_t*>(base + K::OFF_BAR)}; }
  __device__ __forceinline__ volatile int* abort() const { return reinterpret_cast<volatile int*>(base + K::OFF_ABORT); }
  template <typename V>
  __device__ __forceinline__ V* small(int off) const {
    return reinterpret_cast<V*>(base + (OWN ? K::OFF_SMALL_O : K::OFF_SMALL) + group * C::SMALL + off);
  }
  __device__ __forceinline__ unsigned char* pt() const {  // P^T
    return base + (OWN ? K::OFF_PO + group * C::PB : K::OFF_P);
  }
  __device__ __forceinline__ uint32_t s_at() const { return at + (OWN ? K::S_OWN : K::S_COL + C::NG * group); }
  __device__ __forceinline__ uint32_t o_at() const {
    return at + (OWN ? K::O_OWN + group * kOwnRows * K::NDC : K::O_COL + C::NG * group);
  }
  // Every softmax warp of the group arrives and waits (bounded); what was
  // written to shared memory before is visible after.
  __device__ __forceinline__ bool exchange() {
    __syncwarp();
    uint64_t* b = bar().template xch<OWN>(group);
    if ((threadIdx.x & 31) == 0) mbar_arrive(b);
    const bool ok = wait(b, xc & 1, abort());
    ++xc;
    return __all_sync(0xffffffffu, ok);
  }
};

// One visit of a segment: its tiles' softmax, then the partial result.  The
// rows' references live in shared memory; a tile only exchanges whether any
// score outgrew its row's, which after a visit's first tile is rare (it also
// happens when a window first lets a row see a key).
template <int D, int NP, bool OWN, typename Walk>
__device__ bool softmax_visit(const SharedParams& p, Walk& w, SoftCtx<D, NP, OWN>& c) {
  using C = typename SoftCtx<D, NP, OWN>::C;
  constexpr int N = OWN ? kOwnRows : NP, NDC = (D + 127) / 128, NG = C::NG;
  const SharedGeom& g = p.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q4 = warp & 3, t = 32 * q4 + lane;
  const int row0 = OWN ? 0 : NG * c.group;  // this warpgroup's first row of the block
  const float sl2 = g.scale * kLog2e;
  float* red = c.template small<float>(C::RED);
  float* thr = c.template small<float>(C::THR);
  float* use = c.template small<float>(C::USE);
  float* alp = c.template small<float>(C::ALPHA);
  int2* rng = c.template small<int2>(C::RNG);
  int* bnd = c.template small<int>(C::BND);
  volatile int* grow_tag = bnd + 8;   // [2] tile (plus one) at which some score outgrew its reference
  volatile int* scale_tag = bnd + 10;  // [1] tile (plus one) at which some row with earlier keys did
  const int blk = w.blk, slot = w.slot;

  // visible keys of row t (own cache: own indices), and bounds over all rows
  {
    int lo = 0, hi = INT32_MAX;  // rows that are no query mask nothing: their columns are never read
    bool row = false;
    if (t < NG) {
      const int r = row0 + t;  // row of the block
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
  if (!c.exchange()) return false;
  const int lo_all = max(max(bnd[0], bnd[2]), max(bnd[4], bnd[6]));
  const int hi_all = min(min(bnd[1], bnd[3]), min(bnd[5], bnd[7]));

  float l_part[NG], m_row = -INFINITY;  // thread t < NG holds row t's reference
#pragma unroll
  for (int q = 0; q < NG; ++q) l_part[q] = 0.f;

  bool more = true;
#pragma unroll 1
  while (more) {
    const int n = c.k, buf = c.n & 1, key0 = w.key0();
    const bool first = w.first;
    more = !w.last();
    if (!__all_sync(0xffffffffu, wait(c.bar().template s_full<OWN>(c.group) + buf, (c.sph >> buf) & 1, c.abort()))) return false;
    c.sph ^= 1u << buf;
    tc_fence_after();
    uint32_t sr[NG];
    if constexpr (NG == 16) tmem_ld16(c.s_at() + N * buf, sr);
    else tmem_ld32(c.s_at() + N * buf, sr);
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
      if (!c.exchange()) return false;
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
      if (!c.exchange()) return false;
      if (t < NG) {
        const float tm = fmaxf(fmaxf(rb[t], rb[NG + t]), fmaxf(rb[2 * NG + t], rb[3 * NG + t]));
        float a = 1.f;
        if (tm > m_row) {
          const float up = tm + kRoomLog2;
          if (m_row != -INFINITY) {
            a = fast_exp2(m_row - up);
            *scale_tag = n + 1;
          }
          m_row = up;
          use[t] = up;
          thr[t] = up;
        } else if (first) {
          use[t] = 0.f;  // no visible key yet
        }
        alp[t] = a;
      }
      if (!c.exchange()) return false;
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
    if (n > 0 && !__all_sync(0xffffffffu, wait(c.bar().template o_done<OWN>(c.group), (n - 1) & 1, c.abort()))) return false;
    if (scale) {  // uniform over the warpgroup
      tc_fence_after();
#pragma unroll 1
      for (int i = 0; i < NDC * (NG / 16); ++i) {
        const int q0 = NG == 16 ? 0 : 16 * (i & 1);
        const uint32_t o_at = c.o_at() + N * (NG == 16 ? i : i >> 1) + q0;
        uint32_t ov[16];
        tmem_ld16(o_at, ov);
        tmem_wait_ld();
#pragma unroll
        for (int q = 0; q < 16; ++q) ov[q] = __float_as_uint(__uint_as_float(ov[q]) * alp[q0 + q]);
        tmem_st16(o_at, ov);
      }
      tmem_wait_st();
    }
    unsigned char* pb = c.pt();
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
    if (lane == 0) mbar_arrive(c.bar().template p_full<OWN>(c.group));
    ++c.n;
    ++c.k;
    w.next();
  }

  // the visit's partial: row sums over the 128 threads, then O^T
  float* rb = red + (c.xc & 1) * 4 * NG;
  column_reduce<NG, false>(l_part, lane);
  column_post<NG>(l_part, rb + q4 * NG, lane);
  if (!c.exchange()) return false;
  if (!__all_sync(0xffffffffu, wait(c.bar().template o_done<OWN>(c.group), (c.k - 1) & 1, c.abort()))) return false;
  tc_fence_after();
  const int stride = OWN ? p.s.orow : p.s.prow;  // rows of a slot
  int rows;                                      // of which this segment has, and this group from row NG * group on
  if (OWN) rows = min(kOwnRows, g.M - blk * kOwnRows);
  else if (p.s.nmb > 1) rows = min(N, g.M - blk % p.s.nmb * N);
  else rows = min(p.s.nb, g.B - blk * p.s.nb) * g.M;
  rows -= row0;
  const size_t at = (size_t)slot * stride + row0;
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
      tmem_ld16(c.o_at() + N * h + q0, ov);  // warp-collective
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

// The roles' parts of one phase: `total` tiles from walk `w0` on.  Each role
// goes from the prefix to the own caches by itself, so the ring never empties
// in between (3 us a CTA that had work in both, when they met there).
//
// The TMA producer.  `issued`: slots loaded since the kernel began; nq: the
// phase's blocks of queries.
template <int D, int N, bool OWN, typename Walk>
__device__ __forceinline__ bool produce(const SharedParams& p, unsigned char* base, const Bars& bar, volatile int* abort,
                                        const CUtensorMap* tmQ, const CUtensorMap* tmK, const CUtensorMap* tmV,
                                        const Walk& w0, int total, int& issued, int& nq) {
  using K = ShKernel<D, N>;
  constexpr int NCH = K::NCH, CPS = K::CPS, SPT = K::SPT, NSLOT = K::NSLOT, QD = OWN ? 2 : 1;
  constexpr int AHEAD = OWN ? K::OWN_AHEAD : NSLOT;
  const SharedGeom& g = p.g;
  Walk wk = w0, wv = w0;
  // Own caches, which a call reads once, are the first to leave L2, so that the
  // partials stay there (32 of up to 1,024 keys, D = 256: 48.5 us, else 50.9), and
  // so is a prefix of which a call sees more than a quarter of L2: 64 requests of
  // D = 512 over 268 MB take 103.5 us, else 110.6 (after 256 MB of other data, as
  // between a model's steps, 109.5 and 113.8).  A smaller one may find part of
  // itself again: three prefixes of 17 MB in turn, 32 requests, D = 128, 14.4 us,
  // else 15.8; windows that see 17 of 67 MB, D = 256, 47.0, else 47.5.  At 34 MB the
  // two meet: 17.2 us kept and 18.7 on one prefix over and over, 19.2 and 19.0 on
  // three in turn.  After other data all of 17 to 67 MB are within 1 % either way.
  const uint64_t policy = l2_policy(OWN || p.prefix_pass);
  auto load_tile = [&](Walk& w, const CUtensorMap* m) -> bool {
    const int key0 = w.key0();
    int head = w.h;
    if constexpr (OWN) head += w.b * g.Hkv;
#pragma unroll 1
    for (int sp = 0; sp < SPT; ++sp, ++issued) {
      const int s = issued % NSLOT, old = issued - AHEAD;  // the load that has to have been used
      if (old >= 0 && !wait(bar.slot_empty(old % NSLOT), (old / NSLOT) & 1, abort)) return false;
      mbar_arrive_expect_tx(bar.slot_full(s), K::SLOT);
      tma_load_4d(base + s * K::SLOT, m, bar.slot_full(s), 0, key0, sp * CPS, head, policy);
    }
    w.next();
    return true;
  };
  auto load_k = [&]() -> bool {
    if (wk.first) {
      const int s = nq % QD;
      if (nq >= QD && !wait(bar.q_empty<OWN>(s), ((nq / QD) & 1) ^ 1, abort)) return false;
      mbar_arrive_expect_tx(bar.q_full<OWN>(s), OWN ? K::B::QB : NCH * p.s.prow * 128);
      if constexpr (OWN) {
        tma_load_4d(base + K::OFF_QO + s * K::B::QB, tmQ, bar.q_full<OWN>(s), 0, wk.blk * kOwnRows, 0, wk.b * g.Hkv + wk.h);
      } else {
#pragma unroll 1
        for (int c = 0; c < NCH; ++c)
          tma_load_5d(base + K::OFF_Q + c * N * 128, tmQ, bar.q_full<OWN>(s), 0, wk.blk % p.s.nmb * N, c, wk.h,
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
  return ok;
}

// The MMA issuer.  `used`: slots consumed since the kernel began.
template <int D, int NP, bool OWN, typename Walk>
__device__ __forceinline__ bool multiply(const SharedParams& p, unsigned char* base, const Bars& bar, volatile int* abort,
                                         uint32_t tmem, const Walk& w0, int total, int& used) {
  using K = ShKernel<D, NP>;
  using C = typename std::conditional<OWN, typename K::B, typename K::A>::type;
  constexpr int N = OWN ? kOwnRows : NP, CPS = K::CPS, SPT = K::SPT, NSLOT = K::NSLOT, QD = OWN ? 2 : 1;
  const uint32_t idS = idesc_f16(T, N, 1, 1, 0, 0);                // K x Q^T, both K-major
  const uint32_t idPV = idesc_f16(T, N, 1, 1, 1, N > 16 ? 1 : 0);  // V^T (MN-major) x P^T
  const uint32_t s_at = tmem + (OWN ? K::S_OWN : K::S_COL), o_at = tmem + (OWN ? K::O_OWN : K::O_COL);
  Walk ws = w0, wv = w0;
  int nq = 0, gs = 0, gv = 0;  // own: the warpgroup of the walks' visits
  uint32_t pph = 0;            // phases of p_full
  auto issue_s = [&](int n) -> bool {  // S^T(n) into buffer n & 1
    const int qs = nq % QD;
    if (ws.first && !wait(bar.q_full<OWN>(qs), (nq / QD) & 1, abort)) return false;
    uint64_t qd = smem_desc_sw128(smem_u32(base + (OWN ? K::OFF_QO : K::OFF_Q) + qs * C::QB), 16, 1024);
#pragma unroll 1
    for (int sp = 0; sp < SPT; ++sp, ++used) {
      const int s = used % NSLOT;
      if (!wait(bar.slot_full(s), (used / NSLOT) & 1, abort)) return false;
      tc_fence_after();
      uint64_t kd = smem_desc_sw128(smem_u32(base + s * K::SLOT), 16, 1024);
#pragma unroll 1
      for (int cc = 0; cc < CPS; ++cc) {
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          mma_ss(s_at + N * (n & 1), desc_add(kd, ks * 32), desc_add(qd, ks * 32), idS, (sp | cc | ks) ? 1u : 0u);
        kd = desc_add(kd, T * 128);
        qd = desc_add(qd, N * 128);
      }
      mma_commit(bar.slot_empty(s));
    }
    mma_commit(bar.s_full<OWN>(gs) + (n & 1));
    if (ws.last()) {  // the visit's queries are read
      mma_commit(bar.q_empty<OWN>(qs));
      ++nq;
      if (OWN) gs ^= 1;
    }
    ws.next();
    return true;
  };
#pragma unroll 1
  for (int n = -2; n < total; ++n) {
    if (n >= 0) {
      if (!wait(bar.p_full<OWN>(gv), (pph >> gv) & 1, abort)) return false;
      pph ^= 1u << gv;
      tc_fence_after();
      const uint32_t acc = wv.first ? 0u : 1u, o = o_at + (OWN ? gv * kOwnRows * K::NDC : 0);
      const uint64_t pd = smem_desc_sw128(smem_u32(base + (OWN ? K::OFF_PO + gv * C::PB : K::OFF_P)), N > 16 ? T * 128 : 16, 1024);
      // O^T block h (head-dim columns [128 h, 128 h + 128)) += V^T . P^T: one slot a block
#pragma unroll 1
      for (int h = 0; h < SPT; ++h, ++used) {
        const int s = used % NSLOT;
        if (!wait(bar.slot_full(s), (used / NSLOT) & 1, abort)) return false;
        tc_fence_after();
        const uint64_t vd = smem_desc_sw128(smem_u32(base + s * K::SLOT), T * 128, 1024);  // MN-major
#pragma unroll
        for (int ks = 0; ks < T / 16; ++ks)
          mma_ss(o + N * h, desc_add(vd, ks * 2048),
                 N > 16 ? desc_add(pd, ks * 2048) : desc_add(pd, (ks >> 2) * kOwnRows * 128 + (ks & 3) * 32), idPV,
                 (acc || ks > 0) ? 1u : 0u);
        mma_commit(bar.slot_empty(s));
      }
      mma_commit(bar.o_done<OWN>(gv));
      if (OWN && wv.last()) gv ^= 1;
      wv.next();
    }
    if (n + 2 < total && !issue_s(n + 2)) return false;  // after PV(n): S buffer n & 1 is free
  }
  return true;
}

template <int D, int NP>
__global__ void __launch_bounds__(ShKernel<D, NP>::BOUND, 1)
    shared_kernel(const __grid_constant__ CUtensorMap tmQP, const __grid_constant__ CUtensorMap tmQO,
                  const __grid_constant__ CUtensorMap tmKP, const __grid_constant__ CUtensorMap tmVP,
                  const __grid_constant__ CUtensorMap tmKO, const __grid_constant__ CUtensorMap tmVO,
                  const __grid_constant__ SharedParams p) {
  using K = ShKernel<D, NP>;
  using A = typename K::A;
  using B = typename K::B;
  constexpr int THR = K::THREADS, NW = THR / 32;
  extern __shared__ unsigned char smem_raw[];
  __shared__ int scan_sum[NW], scan_min[NW], start_b, start_r;
  __shared__ int4 scan_best[NW];
  unsigned char* base = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const Bars bar{reinterpret_cast<uint64_t*>(base + K::OFF_BAR)};
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar.b + 48);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(base + K::OFF_ABORT);

  const SharedGeom& g = p.g;
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    prefetch_tmap(&tmKP);
    prefetch_tmap(&tmKO);
  }
  if (threadIdx.x < Bars::kCount) {
    mbar_init(bar.b + threadIdx.x, Bars::arrivals(threadIdx.x, K::GROUPS));
    fence_mbar_init();
  }
  // rows of the prefix query block that no box fills stay zero
#pragma unroll 1
  for (int i = threadIdx.x; i < A::QB / 16; i += THR) reinterpret_cast<uint4*>(base + K::OFF_Q)[i] = make_uint4(0, 0, 0, 0);
  if (threadIdx.x < 4 * (K::GROUPS + 2)) {  // the warpgroups' tags
    const int grp = threadIdx.x >> 2;
    unsigned char* small = grp < K::GROUPS ? base + K::OFF_SMALL + grp * A::SMALL + A::BND
                                           : base + K::OFF_SMALL_O + (grp - K::GROUPS) * B::SMALL + B::BND;
    reinterpret_cast<int*>(small)[8 + (threadIdx.x & 3)] = 0;
  }
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
  int nt0;  // tiles of request threadIdx.x
  {
    const int len = threadIdx.x < g.B ? p.own_len[threadIdx.x] : -1;
    int mn = len >= 0 ? min(len, g.own_rows) : INT32_MAX;
    nt0 = own_tiles(g, len);
    int sum = nt0;
#pragma unroll 1
    for (int b = THR + threadIdx.x; b < g.B; b += THR) {
      const int n = p.own_len[b];
      sum += own_tiles(g, n);
      if (n >= 0) mn = min(mn, min(n, g.own_rows));
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
  // Ranges: the number that makes the longest CTA's time shortest.  Pieces go to
  // the CTAs in rounds, the first `rich` CTAs have k of them and the others one
  // less; the own units either level all CTAs (qa for a rich one) or, where the
  // others are done with all of them as soon, stay with those (qb each).
  const int most = nseg ? min(tp, p.most) : 1;
  static_assert(THR >= kPieces, "one candidate a thread");
  if (32 * warp < most) {
    const int i = min(1 + (int)threadIdx.x, most);
    const int np = nseg * i, k = (np + ctas - 1) / ctas, rich = np - (k > 0 ? k - 1 : 0) * ctas, t = tp / i;
    const float pl = k > 0 ? (float)(K::WP * (t + (t * i < tp)) + K::VP) : 0.f, kp = k * pl;
    const float even = (K::WO * (float)own_units + (float)nseg * (K::WP * (float)tp + (float)(K::VP * i))) * (1.f / ctas);
    const int level = rich == ctas ? (own_units + ctas - 1) / ctas : (int)ceilf(fmaxf(0.f, even - kp) * (1.f / K::WO));
    const int alone = rich == ctas ? 0 : (own_units + ctas - rich - 1) / (ctas - rich);
    const float both = kp + K::WV + (float)K::WO * (float)level;
    const float apart = rich == ctas ? INFINITY : fmaxf(kp, kp - pl + K::WV + (float)K::WO * (float)alone);
    const bool join = level > 0 && both < apart;
    const float cost = own_units == 0 ? kp : (join ? both : apart);
    const unsigned mine = (unsigned)fminf(cost, 4.0e6f) << 9 | i, least = __reduce_min_sync(0xffffffffu, mine);
    if (mine == least) scan_best[warp] = make_int4((int)least, join ? level : 0, alone, t);  // (equal where i is)
  }
  __syncthreads();
  int4 best = scan_best[0];
#pragma unroll 1
  for (int i = 1; 32 * i < most; ++i) {
    const int4 v = scan_best[i];
    if ((unsigned)v.x < (unsigned)best.x) best = v;
  }
  const int ns = best.x & 511, pieces = nseg * ns;
  const int rounds = (pieces + ctas - 1) / ctas, rich = pieces - (rounds > 0 ? rounds - 1 : 0) * ctas;
  const int per = best.w, extra = tp - ns * per;  // tiles of a piece, and how many have one more
  const int qa = best.y;                          // own units of a rich CTA, and (qb) of another
  int qb = best.z;
  if (qa > 0) qb = rich == ctas ? 0 : (own_units - min(own_units, rich * qa) + ctas - rich - 1) / (ctas - rich);
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
      const int nt = c0 == 0 ? nt0 : (b < g.B ? own_tiles(g, p.own_len[b]) : 0);
      int inc = nt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      if (c0 > 0) __syncthreads();  // (before the first, scan_best's)
      if (lane == 31) scan_sum[warp] = inc;
      __syncthreads();
      int off = before + inc - nt;
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        const int v = scan_sum[i];
        if (i < warp) off += v;
        before += v;
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
  PrefixWalk wp;
  int total = 0;  // tiles of this CTA's pieces
  if (cta < pieces) {
    wp.p = &p;
    wp.splits = ns;
    wp.tiles = per;
    wp.extra = extra;
    wp.key_lo = key_lo;
#pragma unroll 1
    for (int i = cta; i < pieces; i += ctas) {
      wp.begin(i);
      total += wp.t1 - wp.t;
    }
    wp.begin(cta);
  }
  auto own_walk = [&]() {
    OwnWalk w;
    w.p = &p;
    w.begin(start_b, start_r, o1 - o0);
    return w;
  };
  if (warp == 0) {
    if (elect_one()) {
      int issued = 0, nqa = 0, nqb = 0;
      bool ok = total == 0 || produce<D, NP, false>(p, base, bar, abort_flag, &tmQP, &tmKP, &tmVP, wp, total, issued, nqa);
      if (ok && o0 < o1) {
        // the own queries take over the prefix's bytes once its last scores are formed
        if (K::SHARE_Q && nqa > 0) ok = wait(bar.q_empty<false>(0), (nqa - 1) & 1, abort_flag);
        if (ok) produce<D, NP, true>(p, base, bar, abort_flag, &tmQO, &tmKO, &tmVO, own_walk(), o1 - o0, issued, nqb);
      }
      if (*abort_flag) {  // unwinding: the loads in flight land before shared memory is released
        drain_ring(bar.q_full<false>(0), 1, nqa);
        drain_ring(bar.q_full<true>(0), 2, nqb);
        drain_ring(bar.slot_full(0), K::NSLOT, issued);
      }
    }
  } else if (warp == 1) {
    if (elect_one()) {
      int used = 0;
      const bool ok = total == 0 || multiply<D, NP, false>(p, base, bar, abort_flag, tmem, wp, total, used);
      if (ok && o0 < o1) multiply<D, NP, true>(p, base, bar, abort_flag, tmem, own_walk(), o1 - o0, used);
      mma_commit(bar.drain());
      mbar_wait_drain(bar.drain(), 0);
    }
  } else {
    const int group = (warp - 2) / 4;
    const uint32_t at = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    bool ok = true;
    if (group < K::GROUPS && total > 0) {
      SoftCtx<D, NP, false> c{base, at, group, 0, 0, 0, 0};
#pragma unroll 1
      while (ok && c.n < total) ok = softmax_visit(p, wp, c);
    }
    if (ok && group < 2 && o0 < o1) {  // the own segments in turn
      SoftCtx<D, NP, true> c{base, at, group, 0, 0, 0, 0};
      OwnWalk w = own_walk();
      if (group == 1) c.n += w.skip();
#pragma unroll 1
      while (ok && w.left > 0) {
        ok = softmax_visit(p, w, c);
        if (ok && w.left > 0) c.n += w.skip();
      }
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
// 19.2 and 16.3; 2,048 rows of 6, D = 512: 122 and 119).  AHEAD: at D = 512,
// where a thread's registers bound the rows in flight, 6 (110 us) rather than 8
// (112); in CTAs of 256 threads 4 (15.1 us) rather than 8 (15.6).
template <int D, int THREADS>
__global__ void __launch_bounds__(THREADS) shared_merge_kernel(const __grid_constant__ SharedParams p) {
  constexpr int LANES = D / 4, GR = THREADS / LANES, AHEAD = THREADS == 256 ? 4 : (D == 512 ? 6 : 8);
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
  constexpr int CPS = K::CPS;
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
  const long long nseg = (long long)g.Hkv * s.nrb;
  const long long seen = g.W > 0 && (long long)g.W + g.Lq < g.P ? (long long)g.W + g.Lq : g.P;  // prefix keys, at most
  p.prefix_pass = (double)g.Hkv * seen * D * 4 > 32.0e6;
  p.most = nseg < kPieces ? (int)(kPieces / nseg) : 1;
  auto kern = shared_kernel<D, NP>;
  static std::atomic<unsigned long long> done{0};
  if ((e = allow_smem(kern, (int)K::SMEM, done)) != cudaSuccess) return e;
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
