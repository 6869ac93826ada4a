// Attention of a generation step over a cache held in 8 bits: e4m3 codes with
// one scale for each block of tokens of a head, a length for each request that
// only the device knows.
//
// Request b's keys are k_j = ks_j ck_j and its values v_j = vs_j cv_j (codes ck,
// cv, scales ks, vs of the token's block).  Row i sees the keys of its window, and
//   s_ij = scale ks_j (q_i . ck_j),   o_i = sum_j p_ij vs_j cv_j / sum_j p_ij.
// The scales never meet the codes: ks_j multiplies a finished score, and vs_j goes
// into the weight, w_ij = p_ij vs_j = 2^(y_ij - R_i) with y_ij = s_ij log2 e +
// log2 vs_j and R_i a row's reference.  The row sum is sum_j w_ij / vs_j.
//
// Both products run on the codes as they lie in the cache (kind::f8f6f4), with
// the other operand split so that it keeps its precision.  A bf16 q, scaled by a
// power of two a row, is the exact sum of two e4m3 numbers, q = a + b / 16 (8
// significant bits are 4 and 4), down to 2^-22 of the row's largest element.  A
// weight is rounded to fp16 (half a step: 2^-11) and is there the sum of three
// e5m2 numbers, which are the top bytes of fp16 ones.  The parts are columns of
// one operand, so the codes are read once for all of them, and their products
// are added in fp32.  Turning the codes into bf16 instead would write and read
// each of them twice more in shared memory, in a kernel that has 23 of the
// cache's bytes a clock and SM to take.
//
// Products are transposed: S^T (128 keys x 2 N) = K_tile [a b]^T and O^T (D x 3 N) +=
// V_tile^T [hi mid lo]^T, so that the keys fill the MMA's M dimension whatever the
// number of query rows is.  A block has up to N = 8, 16 or 32 of the G * Lq rows of a
// kv head; a softmax thread has one key of the tile and 8 rows at a time.  Blocks of 16
// and 32 have two groups of four softmax warps, each with half of the rows and with
// barriers of its own, so that one works while the other waits (N = 32, 32 requests over
// up to 8,192 keys, D = 128: 50.4 us with one group and 47.8 with two when they came,
// 36.8 now).
//
// Work.  The unit is one tile of 128 keys of one segment (request, kv head, row
// block), and some for each segment, since a CTA's visit of one takes as long as 1 to 3
// tiles beside them.  The units of all requests, by the device-side lengths, are cut
// into 304 equal runs, one for each CTA, two CTAs an SM.  A segment that lies within
// one run is finished there; one that runs' ends cut leaves a partial (R, sum,
// O) for each run, and a second kernel merges those.  Where a kv head has several
// row blocks, neighbouring CTAs have the same runs of different blocks, so that a
// tile's later reads find it in L2 (16 requests of 32 rows, each over 4,096 keys, D =
// 512: 52.2 us, and 83.2 with the blocks one after the other).
//
// Tiles are aligned to the end of what a request's rows see: one that would
// reach past it starts earlier (below key 0 the TMA fills zeros), so nothing
// behind a request's length is loaded.
//
// Bounds.  Up to 8 rows over long caches by HBM: 32 requests of up to 16,384 tokens, D
// = 512, 153 us, 7.0 TB/s of cache; 64 of up to 8,192, D = 128, 44.0 us, 6.1 TB/s, of
// which some 8 are not the stream's: 0.7 lengths and split, 2.7 until the first tiles
// are there, 1 from the last tile's arrival to a run's end, 1.0 until the merge may
// begin, 1.6 merge, 0.5 until the next call's lengths.  Those are what a short call takes
// (4 requests of up to 1,024, D = 128: 8.0 us, and as much on the host).  At D = 64 the
// softmax of a tile, 0.7 us of a CTA for 8 rows, is as long as its stream (64
// requests of 16 / 2 heads over 16,384 keys: 48.8 us, 5.5 TB/s; three CTAs an SM were
// 2.3 us faster there, and 1 to 4 us slower at the other head dims).  With 9 rows and
// more neither HBM nor the tensor pipe is busy, but the chain of a tile's steps in the
// softmax warps: 32 rows over 16,384 keys, D = 64, issue in 58 % of an SM's cycles with
// DRAM at 31 %; two blocks of 16, D = 512, in 30 % with DRAM at 65 %, L2 at 42 %, half of
// the stalls being on loads and scores (16 requests over 4,096 keys: 52.2 us for 40.2 of
// bytes).
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "swa_internal.h"
#include "tc_ptx.cuh"

namespace swa {
namespace {

using namespace tc;

constexpr int T = 128;       // keys per tile
constexpr int kCtas = 304;   // two an SM
constexpr int kSmemMax = 115584;  // dynamic, a CTA: half of an SM's 228 KB less 1 KB that the system keeps and the static
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// A row's reference lies 2^10 below the largest weight when it is set and moves
// when a weight passes 2^15, so that weights stay within fp16 and e5m2 (2^15.8)
// and the references move seldom.  Below the reference the parts reach down to
// 2^-17 (half a step of the last), 2^-27 of the largest weight or less.
constexpr float kBelow = 10.0f, kTop = 15.0f;
constexpr float kUnset = -3.0e38f;  // reference of a row that has seen no key

struct C8Params {
  Cache8Geom g;
  const uint16_t* q;
  const float *ks, *vs;
  const int* kv_len;
  const float* sinks;  // [Hq] or null
  uint16_t* o;         // bf16 [B, Hq, Lq, D]
  float* lse;          // [B, Hq, Lq]
  int4* cuts;          // [kCtas]: the segment that the begin of the CTA's run cuts (-1: none), its partials, their
                       // first CTA (the others are g.lanes apart) and that one's slot
  float *ml, *po;      // partials [2 kCtas][rows of a block][2] and [..][D]
  int orow;            // rows of a partial's slot
  int* status;
};

// Key tiles of a request that any of its rows sees: of its last W + Lq - 1 keys at
// most.  (A length may be any int: none is subtracted from.)
__device__ __forceinline__ int tiles_of(const Cache8Geom& g, int len) {
  const int n = min(len, g.seen);
  return n > 0 ? (n + T - 1) / T : 0;
}

// a / b, 0 <= a < 2^31, 0 < b: an estimate, the estimate of what it left, and the
// last one.  (A part of the integer division's code: what a CTA runs once is fetched
// at the memory's latency.)
__device__ __forceinline__ int quotient(int a, int b) {
  const float inv = __fdividef(1.f, (float)b);
  int q = (int)((float)a * inv);       // off by 2^-21 of it at most
  int r = a - q * b;
  const int d = (int)((float)r * inv);  // of at most 2^10: off by one at most
  q += d;
  r -= d * b;
  return q + (r >= b) - (r < 0);
}

// The runs that a lane's units are cut into (see Cache8Geom), as equal as whole units
// are: the first `extra` have one more.  Runs behind the units are empty.
struct Runs {
  int base, extra;
  __device__ __forceinline__ Runs(int units, int n) : base(quotient(units, n)), extra(units - base * n) {}
  __device__ __forceinline__ int start(int r) const { return r * base + min(r, extra); }
  __device__ __forceinline__ int of(int u) const {  // whose unit u is
    const int wide = extra * (base + 1);
    return u < wide ? u / (base + 1) : extra + (u - wide) / base;
  }
};

// A segment's units: g.visit of no tile, for what a visit takes but for its tiles
// (queries, the first references, the last product, the output), and its tiles.
__device__ __forceinline__ int units_of(const Cache8Geom& g, int tiles) { return tiles > 0 ? tiles + g.visit : 0; }

// A place in a CTA's run: request, kv head, row block, tile.
struct Walk {
  const C8Params* p;
  int left;      // units from here to the end of the run; none: the run is through
  int lane;      // of row blocks: the walk has blocks lane, lane + g.lanes, ..
  int b, h, blk;
  int t, nt, n;  // tile of the segment, its tiles, the request's length
  bool first;    // first tile of this CTA's visit of the segment
  __device__ __forceinline__ void set_request() {
    n = min(p->kv_len[b], p->g.rows);
    nt = tiles_of(p->g, n);
  }
  __device__ __forceinline__ void begin(int b0, int len, int r, int units) {  // unit r of request b0's
    b = b0;
    n = min(len, p->g.rows);
    nt = tiles_of(p->g, n);
    const int in = quotient(r, nt + p->g.visit), per = blocks();
    t = r - in * (nt + p->g.visit) - p->g.visit;
    h = per == 1 ? in : quotient(in, per);
    blk = lane + p->g.lanes * (in - h * per);
    left = max(units + min(t, 0), 0);
    t = max(t, 0);
    first = true;
  }
  // the lane's blocks of a head (one, where there are no more blocks than CTAs)
  __device__ __forceinline__ int blocks() const {
    return p->g.nmb == p->g.lanes ? 1 : (p->g.nmb - lane + p->g.lanes - 1) / p->g.lanes;
  }
  __device__ __forceinline__ int head() const { return b * p->g.Hkv + h; }
  __device__ __forceinline__ int key0() const { return n - T * (nt - t); }
  __device__ __forceinline__ bool last() const { return left == 1 || t == nt - 1; }
  __device__ __forceinline__ void next() {
    first = false;
    ++t;
    if (--left == 0 || t < nt) return;
    left = max(left - p->g.visit, 0);
    if (left == 0) return;
    first = true;
    t = 0;
    if ((blk += p->g.lanes) < p->g.nmb) return;
    blk = lane;
    if (++h < p->g.Hkv) return;
    h = 0;
    do {  // the next request with keys (there is one while units are left and the lengths stay)
      if (++b >= p->g.B) {
        left = 0;
        return;
      }
      set_request();
    } while (nt == 0);
  }
  __device__ __forceinline__ void skip() {  // to the next visit
    const int k = min(left, nt - t) - 1;
    t += k;
    left -= k;
    next();
  }
};

// The kernel with blocks of NR query rows: 8, 16, or 32 at D <= 128.
template <int D, int NR>
struct C8 {
  static constexpr int GROUPS = NR > 8 ? 2 : 1;   // of four softmax warps, each with a part of the rows:
  static constexpr int NH = NR / 8 / GROUPS;      // so many eights, one after the other
  // warps: TMA, MMA, softmax, and those that prepare queries (rows of 512, 16 requests of 32 rows over up to 4,096 keys:
  // one warp 40.1 us and two 36.4 when visits weighed nothing in the split; 33.0 and 33.7 since); two CTAs of 12 warps
  // have 80 registers a thread, of which blocks of 32 rows spill 5
  static constexpr int HELPER = 2 + 4 * GROUPS, HELPERS = GROUPS, THR = 32 * (HELPER + HELPERS);
  static constexpr int NS = 2 * NR;               // columns of S^T: 8 rows' q in its first part, then in its second
  static constexpr int NP = NR > 8 ? 3 * NR : 32; // of O^T: weights' three parts (see o_col)
  static constexpr int LINE = D < 128 ? D : 128;  // bytes of a key's line in a slot
  static constexpr int NCH = D / LINE;            // slots per tile and tensor; 128-row blocks of O^T
  static constexpr int SLOT = T * LINE;
  static constexpr int QB = NS * D;               // a block of queries
  static constexpr int PB = NP * T;               // weights
  // the softmax groups' small arrays: [4][8] exchanged maxima / sums, references, rescale factors, row ranges, the
  // visit's tiles; and the row factors of four visits
  static constexpr int RED = 0, REF = 128 * NH, ALPHA = REF + 32 * NH, RNG = ALPHA + 32 * NH, PLAN = RNG + 64 * NH, SOFT = PLAN + 16,
                       QFAC = GROUPS * SOFT, SMALL = QFAC + 16 * NR;
  static constexpr int BARS = 256;
  static constexpr int FIT = (kSmemMax - 1024 - 2 * QB - PB - SMALL - BARS) / SLOT;
  static constexpr int NSLOT = FIT > 4 ? (D == 64 ? 8 : 4) : FIT;
  static constexpr int OFF_Q = NSLOT * SLOT, OFF_P = OFF_Q + 2 * QB, OFF_SMALL = OFF_P + PB, OFF_BAR = OFF_SMALL + SMALL;
  static constexpr size_t SMEM = (size_t)OFF_BAR + BARS + 1024;
  static constexpr uint32_t S_COL = 0, O_COL = 2 * NS;  // TMEM columns: S^T twice, O^T's blocks
  static constexpr uint32_t COLS = O_COL + NP * NCH;
  static constexpr uint32_t TCOLS = COLS <= 64 ? 64 : (COLS <= 128 ? 128 : 256);  // (two CTAs share the 512)
  static_assert(COLS <= 256, "TMEM columns");
  static_assert(NSLOT >= 3 && SMEM <= (size_t)kSmemMax, "shared memory");
};

// Columns of an eight's weights (and of their products): the first two parts, and 16 for
// the third parts of two eights between them.
__device__ __forceinline__ int o_col(int eight) { return 48 * (eight >> 1) + 32 * (eight & 1); }
__device__ __forceinline__ int lo_col(int eight) { return 48 * (eight >> 1) + 16 + 8 * (eight & 1); }

// Barriers (words from OFF_BAR on).
struct Bars {
  uint64_t* b;
  __device__ __forceinline__ uint64_t* slot_full(int i) const { return b + i; }       // [8]
  __device__ __forceinline__ uint64_t* slot_empty(int i) const { return b + 8 + i; }  // [8]
  __device__ __forceinline__ uint64_t* q_full(int i) const { return b + 16 + i; }     // [2]
  __device__ __forceinline__ uint64_t* q_empty(int i) const { return b + 18 + i; }    // [2]
  __device__ __forceinline__ uint64_t* s_full(int i) const { return b + 20 + i; }     // [2] S^T in TMEM
  __device__ __forceinline__ uint64_t* p_full() const { return b + 22; }              // weights written (O^T rescaled)
  __device__ __forceinline__ uint64_t* o_done() const { return b + 23; }              // the second product finished
  __device__ __forceinline__ uint64_t* drain() const { return b + 24; }
  static constexpr int kCount = 25;
  static __device__ __forceinline__ int arrivals(int i, int groups) {
    return i == 16 || i == 17 || i == 22 ? 4 * groups : 1;
  }
};

// Shared-memory matrix descriptors: layout 2 is the 128-byte swizzle, 4 the 64-byte one, 0 none.
__device__ __forceinline__ uint64_t smem_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo, uint32_t layout) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)((lbo >> 4) & 0x3FFFu) << 16 |
         (uint64_t)((sbo >> 4) & 0x3FFFu) << 32 | (uint64_t)1 << 46 | (uint64_t)layout << 61;
}
// kind::f8f6f4 with fp32 accumulation; types: 0 e4m3, 1 e5m2.
constexpr uint32_t idesc_f8(int M, int N, int a_type, int b_type, int a_mn, int b_mn) {
  return (1u << 4) | ((uint32_t)a_type << 7) | ((uint32_t)b_type << 10) | ((uint32_t)a_mn << 15) |
         ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Waits for a phase as mbar_wait does, in less code (it stands in some twenty places).
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint32_t t0 = (uint32_t)clock();
  do {
    if (mbar_try_wait(bar, parity)) return true;
  } while (!*abort && (uint32_t)clock() - t0 < 4000000000u);  // ~2 s, within the counter's 32 bits
  *abort = 1;
  return false;
}

// Column reduction of 8 columns over the warp's lanes by halving, into dst[0 .. 7].
template <bool MAX>
__device__ __forceinline__ void column_reduce(float (&v)[8], float* dst, int lane) {
  auto op = [](float a, float b) { return MAX ? fmaxf(a, b) : a + b; };
  int o = 16;
#pragma unroll
  for (int h = 4; h >= 1; h >>= 1, o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < h; ++i) {
      const float give = up ? v[i] : v[i + h], keep = up ? v[i + h] : v[i];
      v[i] = op(keep, __shfl_xor_sync(0xffffffffu, give, o));
    }
  }
#pragma unroll
  for (; o >= 1; o >>= 1) v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
  if (lane % 4 == 0) dst[lane / 4] = v[0];
}

// Queries of one visit as the B operand of the first product: rows 4 w .. 4 w + 3
// of the block by one warp, eight lanes a row; row r's parts go to columns 16 (r / 8)
// + r % 8 and 8 further, and its factor (what its scores are multiplied with, but for the keys'
// scales) to fac[r].  Rows from `rows` on are zero.
template <int D, int NR>
__device__ __forceinline__ void prepare_queries(const C8Params& p, int head, int blk, int rows, unsigned char* dst,
                                                float* fac, int w, int lane) {
  constexpr int V = D / 64;  // vectors of 8 elements a lane
  const int r = 4 * w + (lane >> 3), l8 = lane & 7;
  const uint4* src = reinterpret_cast<const uint4*>(p.q + ((size_t)head * p.g.M + blk * NR + r) * D) + l8;
  auto load = [&](int i) { return r < rows ? src[8 * i] : make_uint4(0, 0, 0, 0); };
  uint4 v[V];
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = load(i);
  uint32_t top = 0;  // max |x| of pairs of bf16 patterns
#pragma unroll
  for (int i = 0; i < V; ++i) {
    top = __vmaxu2(top, __vmaxu2(v[i].x & 0x7FFF7FFFu, v[i].y & 0x7FFF7FFFu));
    top = __vmaxu2(top, __vmaxu2(v[i].z & 0x7FFF7FFFu, v[i].w & 0x7FFF7FFFu));
  }
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
  const float amax = __uint_as_float(max(top << 16, top & 0xFFFF0000u));
  const int e = cache8_scale_exponent(amax, -100);
  const float mul = copysignf(cache8_two_to(-e), p.g.scale);
  constexpr int LINE = C8<D, NR>::LINE, NS = 2 * NR;
#pragma unroll(V <= 2 ? V : 1)
  for (int i = 0; i < V; ++i) {
    const uint4 u = V <= 2 ? v[i] : load(i);  // (a rolled loop reads them again: the code is run once or twice)
    const uint32_t x[4] = {u.x, u.y, u.z, u.w};
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float a = __uint_as_float(x[k] << 16) * mul, b = __uint_as_float(x[k] & 0xFFFF0000u) * mul;
      hi[k] = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
      const float2 h = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)hi[k], __NV_E4M3)));
      lo[k] = __nv_cvt_float2_to_fp8x2(make_float2((a - h.x) * 16.f, (b - h.y) * 16.f), __NV_SATFINITE, __NV_E4M3);
    }
    // K-major rows in the swizzle of their line length
    const int col = (8 * i + l8) * 8, at = col % LINE;
    unsigned char* d = dst + col / LINE * NS * LINE + (at & 15);
    auto put = [&](int row, const uint32_t* q) {
      const int turn = D < 128 ? (row >> 1) & 3 : row & 7;
      *reinterpret_cast<uint2*>(d + row * LINE + (((at >> 4) ^ turn) << 4)) = make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
    };
    put(r + (r & ~7), hi);
    put(r + (r & ~7) + 8, lo);
  }
  // (an infinity's parts are 448, as a finite maximum's may be: its row's factor is
  // NaN, scale + 0 * infinity)
  if (l8 == 0) fac[r] = fmaf(amax, 0.f, fabsf(p.g.scale)) * kLog2e * cache8_two_to(e);
  fence_proxy_async_smem();
}

// 1 / sum and the logsumexp of a finished row, its sink folded in.
__device__ __forceinline__ float finish_row(const float* sink, float ref, float l, float* lse) {
  if (ref == kUnset && l == 0.f) {  // no key
    *lse = sink ? *sink : -INFINITY;
    return 0.f;
  }
  if (sink) return sink_finish(*sink, ref, l, lse);
  *lse = (ref + log2f(l)) * kLn2;
  return 1.f / l;
}

// Barrier of a group's four softmax warps; `any`: whether any of their threads says so.
// Its wait needs no limit: the warps go through all of them whatever their bounded
// waits on the other roles say, and how often is what one thread says to all (a
// visit's tiles), so that lengths that a faulty program changes while the kernel
// runs can make them no different.
__device__ __forceinline__ void soft_sync(int group) {
  if (group == 0) asm volatile("barrier.cta.sync 1, 128;" ::: "memory");
  else asm volatile("barrier.cta.sync 3, 128;" ::: "memory");
}
template <int ID>
__device__ __forceinline__ bool any_of(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, "
      "q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x), "n"(ID)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ bool soft_any(int group, bool x) { return group == 0 ? any_of<1>(x) : any_of<3>(x); }
// The MMA warp has tensor memory, for itself and the softmax warps.
template <int THR>
__device__ __forceinline__ void tmem_sync() {
  asm volatile("barrier.cta.sync 2, %0;" ::"n"(THR) : "memory");
}

// The softmax warps' state over a run.
struct Soft {
  uint32_t at;   // TMEM: this thread's lane
  int n;         // tiles so far: S^T(n) is in buffer n & 1
  int visit;
  int tiles;     // the visit's; none: the run is through
  float ks, vs;  // scales of this thread's key of tile n
};
__device__ __forceinline__ void load_scales(const C8Params& p, const Walk& w, int t, Soft& c) {
  const size_t at = (size_t)w.head() * p.g.nblk + (max(w.key0() + t, 0) >> p.g.lb);
  c.ks = p.ks[at];
  c.vs = p.vs[at];
}

// What a group's warps have to see before a visit (w at its begin, or behind the
// run): the rows' visible keys, no references, the number of tiles.
template <int D, int NR>
__device__ __forceinline__ void plan_visit(const C8Params& p, unsigned char* small, const Walk& w, int t, int r0) {
  using C = C8<D, NR>;
  constexpr int R = 8 * C::NH;
  const Cache8Geom& g = p.g;
  if (t < R) {  // rows that are no query mask nothing: their columns are never read
    const int row = w.blk * NR + r0 + t;
    int lo = 0, hi = INT32_MAX;
    if (row < g.M) {
      hi = w.n - g.Lq + (g.Lq > 1 ? row % g.Lq : 0);
      lo = g.W > 0 ? max(0, hi - g.W + 1) : 0;
    }
    reinterpret_cast<int2*>(small + C::RNG)[t] = make_int2(lo, hi);
    reinterpret_cast<float*>(small + C::REF)[t] = -kUnset;  // (the references' negatives)
  }
  if (t == 0) *reinterpret_cast<int*>(small + C::PLAN) = w.left > 0 ? min(w.left, w.nt - w.t) : 0;
}

// One visit of a segment: its tiles' weights, then the result or the partial.
// After a wait that ran out everything here goes on with what is there, to the
// visit's end: the call's results are then undefined, and its status says so.
template <int D, int NR>
__device__ __forceinline__ void softmax_visit(const C8Params& p, unsigned char* base, const Bars& bar,
                                              volatile int* abort, Walk& w, Soft& c) {
  using C = C8<D, NR>;
  constexpr int NP = C::NP, NH = C::NH, R = 8 * NH;
  const Cache8Geom& g = p.g;
  const int lane = threadIdx.x & 31, q4 = (threadIdx.x >> 5) & 3, t = 32 * q4 + lane;
  const int group = C::GROUPS == 1 ? 0 : threadIdx.x >= 192, r0 = R * group;  // the group's rows: r0 .. r0 + R - 1 of the block's
  unsigned char* small = base + C::OFF_SMALL + group * C::SOFT;
  float* red = reinterpret_cast<float*>(small + C::RED);
  float* nref = reinterpret_cast<float*>(small + C::REF);  // the references' negatives
  float* alp = reinterpret_cast<float*>(small + C::ALPHA);
  int2* rng = reinterpret_cast<int2*>(small + C::RNG);
  const float* fac = reinterpret_cast<const float*>(base + C::OFF_SMALL + C::QFAC) + (c.visit & 3) * NR + r0;
  const int head = w.head(), len = w.n, row0 = w.blk * NR + r0, rows = min(R, g.M - row0);  // (rows < 1: none)
  const bool whole = w.t == 0 && w.left >= w.nt;  // the visit is of the whole segment
  // every row sees the keys from lo_all to hi_all
  const int lo_all = g.W > 0 ? max(0, len - g.W) : 0, hi_all = len - g.Lq;

  uint64_t l_part[R / 2];  // pairs of rows
  float m_row = kUnset;    // thread t < R holds row t's reference
#pragma unroll
  for (int q = 0; q < R / 2; ++q) l_part[q] = 0;

  bool fresh = true;
#pragma unroll 1
  for (int k = 0; k < c.tiles; ++k) {
    const int n = c.n, buf = n & 1, key0 = w.key0();
    const float vscale = fmaxf(c.vs, cache8_two_to(kCache8LeastExponent)), lv = __log2f(vscale);
    const uint64_t ks2 = f2_pack(c.ks, c.ks), lv2 = f2_pack(lv, lv), iv2 = f2_pack(__fdividef(1.f, vscale), __fdividef(1.f, vscale));
    w.next();
    if (w.left > 0) load_scales(p, w, t, c);  // the next tile's are under way meanwhile
    const bool edge = !(key0 >= lo_all && key0 + T - 1 <= hi_all);
    wait(bar.s_full(buf), (n >> 1) & 1, abort);
    __syncwarp();
    tc_fence_after();
#pragma unroll
    for (int hf = 0; hf < NH; ++hf) {  // 8 rows
      uint32_t sc[16];  // 8 rows' products with the first part of q, then with the second
      tmem_ld16(c.at + C::S_COL + C::NS * buf + 16 * (NH * group + hf), sc);
      tmem_wait_ld();
      uint64_t y[4], z[4];
      const uint64_t small16 = f2_pack(0.0625f, 0.0625f);
#pragma unroll
      for (int q = 0; q < 4; q += 2) {
        const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(fac + 8 * hf + 2 * q);
        const uint64_t ff[2] = {f.x, f.y};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = 2 * (q + i);
          const uint64_t a = f2_pack(__uint_as_float(sc[r]), __uint_as_float(sc[r + 1]));
          const uint64_t b = f2_pack(__uint_as_float(sc[8 + r]), __uint_as_float(sc[9 + r]));
          y[q + i] = f2_fma(f2_fma(b, small16, a), f2_mul(ff[i], ks2), lv2);
        }
      }
      if (edge) {
        const int key = key0 + t;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int4 r = *reinterpret_cast<const int4*>(rng + 8 * hf + 2 * q);
          float2 v = f2_unpack(y[q]);
          if (key < r.x || key > r.y) v.x = -INFINITY;
          if (key < r.z || key > r.w) v.y = -INFINITY;
          y[q] = f2_pack(v.x, v.y);
        }
      }
      auto less_reference = [&]() {  // z = y - reference
#pragma unroll
        for (int q = 0; q < 4; q += 2) {
          const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(nref + 8 * hf + 2 * q);
          z[q] = f2_add(y[q], f.x);
          z[q + 1] = f2_add(y[q + 1], f.y);
        }
      };
      bool grow = true;
      if (!fresh) {
        less_reference();
        float over = -INFINITY;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float2 v = f2_unpack(z[q]);
          over = fmax3(over, v.x, v.y);
        }
        grow = soft_any(group, over > kTop);
      }
      if (grow) {  // some weight passes the top, or the visit begins
        float mx[8];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float2 v = f2_unpack(y[q]);
          mx[2 * q] = v.x;
          mx[2 * q + 1] = v.y;
        }
        column_reduce<true>(mx, red + q4 * 8, lane);
        soft_sync(group);
        bool moved = false;
        const int i = t - 8 * hf;
        if (i >= 0 && i < 8) {
          const float tm = fmaxf(fmaxf(red[i], red[8 + i]), fmaxf(red[16 + i], red[24 + i]));
          float a = 1.f;
          if (tm - m_row > kTop) {  // (a row without a key yet: its reference is the lowest number)
            const float to = tm - kBelow;
            if (m_row != kUnset) {
              a = fast_exp2(m_row - to);
              moved = true;
            }
            m_row = to;
            nref[t] = -to;
          }
          alp[t] = a;
        }
        if (soft_any(group, moved)) {  // sums and O^T of these rows move with their references
#pragma unroll
          for (int q = 0; q < 4; ++q) l_part[4 * hf + q] = f2_mul(l_part[4 * hf + q], *reinterpret_cast<const uint64_t*>(alp + 8 * hf + 2 * q));
          wait(bar.o_done(), (n - 1) & 1, abort);  // (the row has earlier keys: n > 0)
          __syncwarp();
          tc_fence_after();
#pragma unroll 1
          for (int j = 0; j < C::NCH; ++j) {
            const uint32_t at = c.at + C::O_COL + NP * j;
            uint32_t ov[16], ow[8];
            tmem_ld16(at + o_col(NH * group + hf), ov);
            tmem_ld8(at + lo_col(NH * group + hf), ow);
            tmem_wait_ld();
#pragma unroll
            for (int q = 0; q < 16; ++q) ov[q] = __float_as_uint(__uint_as_float(ov[q]) * alp[8 * hf + q % 8]);
#pragma unroll
            for (int q = 0; q < 8; ++q) ow[q] = __float_as_uint(__uint_as_float(ow[q]) * alp[8 * hf + q]);
            tmem_st16(at + o_col(NH * group + hf), ov);
            tmem_st8(at + lo_col(NH * group + hf), ow);
          }
          tmem_wait_st();
        }
        less_reference();
      }
      // the weights 2^(y - reference), their row sums, and their three parts: hi is
      // a weight in fp16 rounded to its top byte, mid the rest so, lo the rest of that
      uint32_t part[3][2];
#pragma unroll
      for (int q = 0; q < 4; q += 2) {
        float2 e = f2_unpack(z[q]), f = f2_unpack(z[q + 1]);
        e.x = fast_exp2(e.x);
        e.y = fast_exp2(e.y);
        f.x = fast_exp2(f.x);
        f.y = fast_exp2(f.y);
        uint64_t* l = l_part + 4 * hf + q;
        l[0] = f2_fma(f2_pack(e.x, e.y), iv2, l[0]);
        l[1] = f2_fma(f2_pack(f.x, f.y), iv2, l[1]);
        uint32_t a = pack_half2(e.x, e.y), b = pack_half2(f.x, f.y);
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          const uint32_t ra = a + 0x00800080u, rb = b + 0x00800080u;
          part[i][q / 2] = __byte_perm(ra, rb, 0x7531);
          if (i < 2) {
            const uint32_t ta = ra & 0xFF00FF00u, tb = rb & 0xFF00FF00u;
            const __half2 da = __hsub2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<const __half2*>(&ta));
            const __half2 db = __hsub2(*reinterpret_cast<__half2*>(&b), *reinterpret_cast<const __half2*>(&tb));
            a = *reinterpret_cast<const uint32_t*>(&da);
            b = *reinterpret_cast<const uint32_t*>(&db);
          }
        }
      }
      // the second product of tile n - 1 has finished with the weights' buffer
      if (hf == 0 && n > 0) wait(bar.o_done(), (n - 1) & 1, abort);
      // MN-major operand without swizzle: 16 columns of a key are 16 bytes.  (Columns
      // of rows that the block has not are multiplied as they are and never read.)
      unsigned char* pb = base + C::OFF_P + t * 16;
      *reinterpret_cast<uint4*>(pb + o_col(NH * group + hf) * T) = make_uint4(part[0][0], part[0][1], part[1][0], part[1][1]);
      *reinterpret_cast<uint2*>(pb + lo_col(NH * group + hf) / 16 * T * 16 + lo_col(NH * group + hf) % 16) = make_uint2(part[2][0], part[2][1]);
    }
    fresh = false;
    fence_proxy_async_smem();  // generic writes -> the tensor core's reads
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar.p_full());
    ++c.n;
  }
  ++c.visit;

  // row sums over the 128 threads, then O^T
#pragma unroll
  for (int hf = 0; hf < NH; ++hf) {
    float l[8];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float2 v = f2_unpack(l_part[4 * hf + q]);
      l[2 * q] = v.x;
      l[2 * q + 1] = v.y;
    }
    column_reduce<false>(l, red + q4 * R + 8 * hf, lane);
  }
  soft_sync(group);
  float* mul = alp;  // a whole segment's 1 / sum
  const size_t slot = (size_t)(2 * (blockIdx.y * gridDim.x + blockIdx.x) + (c.visit > 1 ? 1 : 0)) * p.orow + r0;
  if (t < rows) {
    const float l = (red[t] + red[R + t]) + (red[2 * R + t] + red[3 * R + t]);
    if (whole) {
      const int m = row0 + t;
      float lse;
      mul[t] = finish_row(p.sinks ? p.sinks + (head % g.Hkv) * g.G + m / g.Lq : nullptr, m_row, l, &lse);
      p.lse[(size_t)head * g.M + m] = lse;
    } else {
      *reinterpret_cast<float2*>(p.ml + 2 * (slot + t)) = make_float2(m_row, l);
    }
  }
  plan_visit<D, NR>(p, small, w, t, r0);  // the next one's, while the last product is under way
  soft_sync(group);
  c.tiles = *reinterpret_cast<int*>(small + C::PLAN);
  wait(bar.o_done(), (c.n - 1) & 1, abort);
  __syncwarp();
  tc_fence_after();
#pragma unroll 1
  for (int h = 0; h < C::NCH * NH; ++h) {
    const int ch = h / NH, hf = h % NH;
    uint32_t oa[16], ob[8];
    const uint32_t at = c.at + C::O_COL + NP * ch;
    tmem_ld16(at + o_col(NH * group + hf), oa);  // warp-collective
    tmem_ld8(at + lo_col(NH * group + hf), ob);
    tmem_wait_ld();
    const int d = T * ch + t;
    if (d < D) {
      uint16_t* o = p.o + ((size_t)head * g.M + row0 + 8 * hf) * D + d;
      float* po = p.po + (slot + 8 * hf) * D + d;
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (8 * hf + q < rows) {
          const float v = __uint_as_float(oa[q]) + (__uint_as_float(oa[8 + q]) + __uint_as_float(ob[q]));
          if (whole) o[q * D] = __bfloat16_as_ushort(__float2bfloat16_rn(v * mul[8 * hf + q]));
          else po[q * D] = v;
        }
    }
  }
  tc_fence_before();  // ordered before the next visit's first product by its arrival
}

template <int D, int NR>
__global__ void __launch_bounds__(C8<D, NR>::THR, 2)
    cache8_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                  const __grid_constant__ C8Params p) {
  using C = C8<D, NR>;
  constexpr int NSLOT = C::NSLOT, NCH = C::NCH, NS = C::NS, NP = C::NP;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* base = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const Bars bar{reinterpret_cast<uint64_t*>(base + C::OFF_BAR)};
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar.b + 30);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bar.b + 31);
  float* qfac = reinterpret_cast<float*>(base + C::OFF_SMALL + C::QFAC);
  const Cache8Geom& g = p.g;
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, cta = blockIdx.y * gridDim.x + blockIdx.x;

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  if (threadIdx.x < Bars::kCount) {
    mbar_init(bar.b + threadIdx.x, Bars::arrivals(threadIdx.x, C::GROUPS));
    fence_mbar_init();
  }
  __syncthreads();
  // ---- this CTA's run, by every warp for itself: the tiles of all requests, then
  // the request that the run's first unit belongs to.  Gone through twice, first as if
  // all requests were full: code that a CTA runs once is fetched at the memory's
  // latency, and there is time before the predecessor's end.
  Walk first;  // the run's first unit
  first.p = &p;
  first.lane = blockIdx.x;
  const int hn = g.Hkv * first.blocks();
  Runs runs(0, 1);
  int u0 = 0;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    if (pass) {
      grid_dependency_wait();
      // Tensor memory is taken after the predecessor's end and before a dependent
      // may be placed: a grid that held columns while it waits for another that has
      // yet to allocate its own, on the same SM, would wait for ever.
      if (warp == 1) {
        tmem_alloc(tmem_slot, C::TCOLS);
        tmem_relinquish();
        grid_launch_dependents();  // the merge waits for this grid's end
      }
    }
    auto length = [&](int b) { return b >= g.B ? -1 : pass ? p.kv_len[b] : g.rows; };
    const int len0 = length(lane);  // of the first 32
    int all = units_of(g, tiles_of(g, len0));
#pragma unroll 1
    for (int b = lane + 32; b < g.B; b += 32) all += units_of(g, tiles_of(g, length(b)));
    all = __reduce_add_sync(0xffffffffu, all);
    first.left = 0;
    runs = Runs(all * hn, gridDim.y);
    u0 = runs.start(blockIdx.y);
    const int units = runs.start(blockIdx.y + 1) - u0;
    if (units > 0) {
      int before = 0;
#pragma unroll 1
      for (int b0 = 0; b0 < g.B; b0 += 32) {
        const int len = b0 == 0 ? len0 : length(b0 + lane);
        const int own = units_of(g, tiles_of(g, len));
        int inc = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += v;
        }
        const unsigned here = __ballot_sync(0xffffffffu, u0 < (before + inc) * hn);
        if (here) {
          const int l = __ffs(here) - 1;
          const int at = before + __shfl_sync(0xffffffffu, inc - own, l);
          first.begin(b0 + l, __shfl_sync(0xffffffffu, len, l), u0 - at * hn, units);
          break;
        }
        before += __shfl_sync(0xffffffffu, inc, 31);
      }
    }
  }
  const bool any = first.left > 0;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (any && elect_one()) {
      // the cache, which a call reads once (but for further row blocks), gives way in L2
      const uint64_t policy = l2_policy(true);
      Walk wk = first, wv = first;
      int issued = 0;
      auto load_tile = [&](Walk& w, const CUtensorMap* m) -> bool {
        const int key0 = w.key0(), head = w.head();
#pragma unroll 1
        for (int c = 0; c < NCH; ++c, ++issued) {
          const int s = issued % NSLOT;
          if (issued >= NSLOT && !wait(bar.slot_empty(s), ((issued / NSLOT) & 1) ^ 1, abort_flag)) return false;
          mbar_arrive_expect_tx(bar.slot_full(s), C::SLOT);
          tma_load_4d(base + s * C::SLOT, m, bar.slot_full(s), 0, key0, c, head, policy);
        }
        w.next();
        return true;
      };
      // slots in MMA order: K(0), K(1), then per tile n: V(n), K(n + 2)
      bool ok = true;
#pragma unroll 1
      for (int n = -2; ok && wv.left > 0; ++n)
        ok = (n < 0 || load_tile(wv, &tmV)) && (wk.left == 0 || load_tile(wk, &tmK));
      if (*abort_flag) drain_ring(bar.slot_full(0), NSLOT, issued);  // loads in flight land before shared memory is released
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    tmem_sync<32 + 128 * C::GROUPS>();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    if (any && elect_one()) {
      constexpr uint32_t idS = idesc_f8(T, NS, 0, 0, 0, 0);  // K x Q^T, both K-major, e4m3
      constexpr uint32_t idO = idesc_f8(T, NP, 0, 1, 1, 1);  // V^T (e4m3) x weights^T (e5m2), both MN-major
      constexpr uint32_t SWZ = D < 128 ? 4 : 2;
      // 8 lines make a swizzled group.  At D = 64 the second product's rows 64-127 repeat 0-63 and are never read.
      const uint64_t kd0 = smem_desc(smem_u32(base), D < 128 ? 0 : 16, 8 * C::LINE, SWZ);
      const uint64_t qd0 = smem_desc(smem_u32(base + C::OFF_Q), 16, 8 * C::LINE, SWZ);
      const uint64_t pd = smem_desc(smem_u32(base + C::OFF_P), 8 * 16, T * 16, 0);
      Walk ws = first, wv = first;
      int used = 0, nq = 0;
      auto issue_s = [&](int n) -> bool {  // S^T(n)
        const int qs = nq & 1;
        if (ws.first && !wait(bar.q_full(qs), (nq >> 1) & 1, abort_flag)) return false;
#pragma unroll 1
        for (int c = 0; c < NCH; ++c, ++used) {
          const int s = used % NSLOT;
          if (!wait(bar.slot_full(s), (used / NSLOT) & 1, abort_flag)) return false;
          tc_fence_after();
          const uint32_t s_at = tmem + C::S_COL + NS * (n & 1);
          const uint64_t kd = desc_add(kd0, s * C::SLOT), qd = desc_add(qd0, qs * C::QB + c * NS * C::LINE);
#pragma unroll
          for (int k = 0; k < C::LINE / 32; ++k)
            mma_f8(s_at, desc_add(kd, k * 32), desc_add(qd, k * 32), idS, (c | k) ? 1u : 0u);
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
      bool ok = true;
#pragma unroll 1
      for (int n = -2; ok && wv.left > 0; ++n) {
        if (n >= 0) {
          if (!wait(bar.p_full(), n & 1, abort_flag)) break;
          tc_fence_after();
          const uint32_t acc = wv.first ? 0u : 1u;
#pragma unroll 1
          for (int c = 0; c < NCH; ++c, ++used) {
            const int s = used % NSLOT;
            if (!(ok = wait(bar.slot_full(s), (used / NSLOT) & 1, abort_flag))) break;
            tc_fence_after();
            const uint64_t vd = desc_add(kd0, s * C::SLOT);
#pragma unroll
            for (int k = 0; k < T / 32; ++k)
              mma_f8(tmem + C::O_COL + NP * c, desc_add(vd, k * 32 * C::LINE), desc_add(pd, k * 32 * 16), idO,
                     (acc || k > 0) ? 1u : 0u);
            mma_commit(bar.slot_empty(s));
          }
          if (!ok) break;
          mma_commit(bar.o_done());
          wv.next();
        }
        if (ws.left > 0) ok = issue_s(n + 2);  // the weights of tile n have been written: its scores' buffer is free
      }
      mma_commit(bar.drain());
      mbar_wait_drain(bar.drain(), 0);
    }
  } else if (warp < C::HELPER) {
    // ------------------------------------------------------------ softmax
    Walk w = first;
    Soft c;
    c.n = c.visit = 0;
    if (any) {
      load_scales(p, w, 32 * (warp & 3) + lane, c);
      if (warp - 2 < NR / 4)
        prepare_queries<D, NR>(p, w.head(), w.blk, min(NR, g.M - w.blk * NR), base + C::OFF_Q, qfac, warp - 2, lane);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar.q_full(0));
    }
    const int group = (warp - 2) / 4;
    unsigned char* small = base + C::OFF_SMALL + group * C::SOFT;
    plan_visit<D, NR>(p, small, w, 32 * (warp & 3) + lane, 8 * C::NH * group);
    tmem_sync<32 + 128 * C::GROUPS>();
    tc_fence_after();
    c.at = *tmem_slot + ((uint32_t)(32 * (warp & 3)) << 16);
    c.tiles = *reinterpret_cast<int*>(small + C::PLAN);
#pragma unroll 1
    while (c.tiles > 0) softmax_visit<D, NR>(p, base, bar, abort_flag, w, c);
  } else {
    // ------------------------------------------------------------ the later visits' queries
    if (warp == C::HELPER && lane == 0) {  // for the merge
      int4 cut = make_int4(-1, 0, 0, 0);
      if (any && first.t > 0) {
        const int begin = u0 - first.t, c0 = runs.of(begin);  // the segment's first tile
        cut = make_int4(first.head() * g.nmb + first.blk, runs.of(begin + first.nt - 1) - c0 + 1,
                        c0 * g.lanes + first.lane,
                        2 * (c0 * g.lanes + first.lane) + (runs.start(c0) >= begin - g.visit ? 0 : 1));
      }
      p.cuts[cta] = cut;
    }
    Walk w = first;
    if (any) w.skip();
    int filled = NR / 4 * 0x11;  // groups of rows of either buffer that may not be zero
#pragma unroll 1
    for (int v = 1; w.left > 0; ++v) {
      const int s = v & 1;
      if (v >= 2 && !__all_sync(0xffffffffu, wait(bar.q_empty(s), ((v >> 1) & 1) ^ 1, abort_flag))) break;
      // (the softmax reads the factors of visit v - 3 at most: the scores are two tiles ahead of it, the queries two visits)
      const int rows = min(NR, g.M - w.blk * NR);
      // all rows are asked for at once (four at a time would take the memory's latency as often)
      const unsigned char* q = reinterpret_cast<const unsigned char*>(p.q + ((size_t)w.head() * g.M + w.blk * NR) * D);
#pragma unroll 1
      for (int i = threadIdx.x - 32 * C::HELPER; i < rows * (D / 64); i += 32 * C::HELPERS)
        asm volatile("prefetch.global.L1 [%0];" ::"l"(q + 128 * i));
      // rows behind the block's are zero once they have been
      const int groups = (rows + 3) / 4, old = filled >> (4 * s) & 15;  // of four rows
#pragma unroll 1
      for (int i = warp - C::HELPER; i < max(groups, old); i += C::HELPERS)
        prepare_queries<D, NR>(p, w.head(), w.blk, rows, base + C::OFF_Q + s * C::QB, qfac + (v & 3) * NR, i, lane);
      filled = (filled & ~(15 << (4 * s))) | groups << (4 * s);
      __syncwarp();
      if (lane < 4 * C::GROUPS / C::HELPERS) mbar_arrive(bar.q_full(s));
      w.skip();
    }
    // requests without a key: no unit is theirs
#pragma unroll 1
    for (int b = cta; warp == C::HELPER && b < g.B; b += gridDim.x * gridDim.y) {
      const int len = p.kv_len[b];
      if (len < 0 || tiles_of(g, len) > 0) continue;
      const size_t at = (size_t)b * g.Hkv * g.M;
      const int rows = g.Hkv * g.M;
      for (int r = lane; r < rows; r += 32) p.lse[at + r] = p.sinks ? p.sinks[r / g.Lq] : -INFINITY;
      uint4* o = reinterpret_cast<uint4*>(p.o + at * D);
      for (long long i = lane; i < (long long)rows * (D / 8); i += 32) o[i] = make_uint4(0, 0, 0, 0);
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (*abort_flag && threadIdx.x == 0) atomicCAS(p.status, 0, kStatusTimeout);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(*tmem_slot, C::TCOLS);
  }
}

// Merge of the partials of the segment that the begin of run blockIdx.x cuts.  A
// segment in n runs has n - 1 cuts, whose CTAs take its rows in turn, or pieces of
// 64 columns of its rows where there are more cuts than those; a CTA's warps share
// the partials of its pieces.  With R = max R_i over the partials,
// o = sum 2^(R_i - R) O_i / sum 2^(R_i - R) l_i.
constexpr int kMergeWarps = 4, kMergeSides = 2;  // warps a CTA, CTAs a cut

// One pass over a CTA's pieces of W columns; n = 0: none (see the kernel).
template <int D, int W>
__device__ __forceinline__ void merge_pieces(const C8Params& p, const int4& cut, int rows, float (&part)[kMergeWarps][W],
                                             float2 (&stat)[kMergeWarps]) {
  constexpr int LANES = W / 4 < 32 ? W / 4 : 32, SIDE = 32 / LANES;  // lanes on a partial, partials side by side
  constexpr int N = W / 4 / LANES, AHEAD = 4 / N, PIECES = D / W;    // vectors a lane, partials under way, pieces of a row
  const Cache8Geom& g = p.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l0 = lane % LANES;
  const int n = cut.y, head = g.nmb == 1 ? cut.x : cut.x / g.nmb, blk = cut.x - head * g.nmb;
  const int apart = g.lanes == 1 ? (int)blockIdx.x - cut.z : ((int)blockIdx.x - cut.z) / g.lanes;  // runs
  // pieces first, first + step, .. of `all` (the quotient of numbers below 2^12 is exact)
  const int all = rows * PIECES, first = kMergeSides * (apart - 1) + blockIdx.y, step = max(kMergeSides * (n - 1), 1);
  const int mine = n == 0 ? 4 : (first < all ? (int)__fdividef(all - first + step - 0.5f, (float)step) : 0);
  static_assert(kMergeWarps == 4, "the next line");
  const int sh = mine > 2 ? 0 : (mine == 2 ? 1 : 2), share = 1 << sh;  // warps on a piece
  const int k = warp & (share - 1);
#pragma unroll 1
  for (int i0 = 0; i0 < mine; i0 += kMergeWarps >> sh) {
    const int i = i0 + (warp >> sh);
    const bool on = i < mine;
    const int piece = first + i * step, row = piece / PIECES, col = (piece - row * PIECES) * W;
    float acc[4 * N];
#pragma unroll
    for (int e = 0; e < 4 * N; ++e) acc[e] = 0.f;
    float m = kUnset, l = 0.f;
    if (on) {
      float4 v[AHEAD][N];
      float2 ml[AHEAD];
      auto load = [&](int a, int j) {
        ml[a] = make_float2(kUnset, 0.f);
        if (j >= n) return;
        const size_t at = (size_t)(j == 0 ? cut.w : 2 * (cut.z + j * g.lanes)) * p.orow + row;
        ml[a] = *reinterpret_cast<const float2*>(p.ml + 2 * at);
        const float4* src = reinterpret_cast<const float4*>(p.po + at * D + col) + l0;
#pragma unroll
        for (int e = 0; e < N; ++e) v[a][e] = src[LANES * e];
      };
      const int j0 = k * SIDE + lane / LANES, dj = share * SIDE;
#pragma unroll 1
      for (int j = j0; j - j0 % dj < max(n, 1); j += dj * AHEAD) {
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) load(a, j + dj * a);
        float to = m;
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) to = fmaxf(to, ml[a].x);
        const float w0 = fast_exp2(m - to);
        l *= w0;
#pragma unroll
        for (int e = 0; e < 4 * N; ++e) acc[e] *= w0;
#pragma unroll
        for (int a = 0; a < AHEAD; ++a)
          if (j + dj * a < n) {  // (a part without a visible key: its sum and O are 0)
            const float w = fast_exp2(ml[a].x - to);
            l = fmaf(w, ml[a].y, l);
#pragma unroll
            for (int e = 0; e < 4 * N; ++e) acc[e] = fmaf(w, reinterpret_cast<const float*>(v[a])[e], acc[e]);
          }
        m = to;
      }
    }
    auto join = [&](float m2, float l2, auto&& of) {  // with another stream's reference, sum and elements
      const float to = fmaxf(m, m2), a = fast_exp2(m - to), b = fast_exp2(m2 - to);
      m = to;
      l = l * a + l2 * b;
#pragma unroll
      for (int e = 0; e < 4 * N; ++e) acc[e] = acc[e] * a + of(e) * b;
    };
    if (SIDE == 2) {
      const float m2 = __shfl_xor_sync(0xffffffffu, m, 16), l2 = __shfl_xor_sync(0xffffffffu, l, 16);
      join(m2, l2, [&](int e) { return __shfl_xor_sync(0xffffffffu, acc[e], 16); });
    }
    auto place = [&](int e) { return 4 * LANES * (e / 4) + 4 * l0 + e % 4; };  // of a lane's element e
    if (share > 1) {
      if (lane == 0) stat[warp] = make_float2(m, l);
#pragma unroll
      for (int e = 0; e < 4 * N; ++e)
        if (lane < LANES) part[warp][place(e)] = acc[e];
      __syncthreads();
      if (on && k == 0) {
#pragma unroll 1
        for (int w = warp + 1; w < warp + share; ++w) join(stat[w].x, stat[w].y, [&](int e) { return part[w][place(e)]; });
      }
      __syncthreads();
    }
    if (!on || k > 0 || lane >= LANES || n == 0) continue;
    const int r = blk * g.nr + row;
    float lse;
    const float inv = finish_row(p.sinks ? p.sinks + (head % g.Hkv) * g.G + r / g.Lq : nullptr, m, l, &lse);
    const size_t at = (size_t)head * g.M + r;
#pragma unroll
    for (int e = 0; e < 4 * N; e += 4) {
      const __nv_bfloat162 x = __floats2bfloat162_rn(acc[e] * inv, acc[e + 1] * inv);
      const __nv_bfloat162 y = __floats2bfloat162_rn(acc[e + 2] * inv, acc[e + 3] * inv);
      *reinterpret_cast<uint2*>(p.o + at * D + col + place(e)) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
    }
    if (col == 0 && lane == 0) p.lse[at] = lse;
  }
}

// What is behind the wait for the main grid is gone through once before it, on no
// partials: code that a CTA runs once is fetched at the memory's latency, and there
// is time while the last runs end.
template <int D>
__global__ void __launch_bounds__(32 * kMergeWarps, 6) cache8_merge_kernel(const __grid_constant__ C8Params p) {
  constexpr int W = D < 256 ? D : 256;  // columns of a piece where there are few cuts
  __shared__ union {
    float whole[kMergeWarps][W], piece[kMergeWarps][64];
  } part;
  __shared__ float2 stat[kMergeWarps];
  grid_launch_dependents();
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    int4 cut = make_int4(0, 0, 0, 0);
    if (pass) {
      grid_dependency_wait();
      cut = p.cuts[blockIdx.x];
      if (cut.x < 0) return;
    }
    const int blk = p.g.nmb == 1 ? 0 : cut.x % p.g.nmb, rows = min(p.g.nr, p.g.M - blk * p.g.nr);
    const bool pieces = D == 64 || cut.y > rows * (D / 64);
    if (pieces || !pass) merge_pieces<D, 64>(p, cut, rows, part.piece, stat);
    if (D > 64 && !pieces) merge_pieces<D, W>(p, cut, rows, part.whole, stat);
  }
}

struct C8Ws {
  size_t cuts, ml, po, total;
};
int slot_rows(const Cache8Geom& g) { return g.M < g.nr ? g.M : g.nr; }
// Key tiles of a request, at most.
long long tiles_most(const Cache8Geom& g) { return ((long long)g.seen + T - 1) / T; }
C8Ws c8_ws(const Cache8Geom& g) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t rows = (size_t)2 * kCtas * slot_rows(g);
  C8Ws w;
  w.cuts = 0;
  w.ml = up(kCtas * sizeof(int4));
  w.po = w.ml + up(rows * 8);
  w.total = w.po + up(rows * g.D * 4);
  return w;
}

// Codes [heads, rows, D] in slots of 128 keys and up to 128 bytes of each: coordinates (0, key, chunk, head).
cudaError_t make_tmap_codes(CUtensorMap* m, const void* ptr, int D, int rows, int heads) {
  const int line = D < 128 ? D : 128;
  const cuuint64_t dims[4] = {(cuuint64_t)line, (cuuint64_t)rows, (cuuint64_t)(D / line), (cuuint64_t)heads};
  const cuuint64_t strides[3] = {(cuuint64_t)D, (cuuint64_t)line, (cuuint64_t)D * rows};
  const cuuint32_t box[4] = {(cuuint32_t)line, T, 1, 1};
  return make_tmap_u8_4d(m, ptr, dims, strides, box, D < 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int D, int NR>
cudaError_t cache8_d(const Cache8Geom& g, const Cache8Args& a, void* ws, int* status, cudaStream_t st) {
  using C = C8<D, NR>;
  CUtensorMap tk, tv;
  cudaError_t e;
  if ((e = make_tmap_codes(&tk, a.k, D, g.rows, g.B * g.Hkv)) != cudaSuccess) return e;
  if ((e = make_tmap_codes(&tv, a.v, D, g.rows, g.B * g.Hkv)) != cudaSuccess) return e;
  const C8Ws w = c8_ws(g);
  unsigned char* wb = static_cast<unsigned char*>(ws);
  C8Params p;
  p.g = g;
  p.q = a.q;
  p.ks = a.ks;
  p.vs = a.vs;
  p.kv_len = a.kv_len;
  p.sinks = a.sinks;
  p.o = a.o;
  p.lse = a.lse;
  p.cuts = reinterpret_cast<int4*>(wb + w.cuts);
  p.ml = reinterpret_cast<float*>(wb + w.ml);
  p.po = reinterpret_cast<float*>(wb + w.po);
  p.orow = slot_rows(g);
  p.status = status;
  auto kern = cache8_kernel<D, NR>;
  static std::atomic<unsigned long long> done{0};
  if ((e = allow_smem(kern, (int)C::SMEM, done)) != cudaSuccess) return e;
  const dim3 grid((unsigned)g.lanes, (unsigned)(kCtas / g.lanes));  // a run's lanes are neighbours
  // both are programmatic dependents of what runs before them: the main grid's
  // set-up and the merge's placement fall into its predecessor's end
  if ((e = launch_dependent(kern, grid, dim3(C::THR), C::SMEM, st, tk, tv, p)) != cudaSuccess) return e;
  if (tiles_most(g) == 1) return cudaSuccess;  // a segment of one tile is not cut
  return launch_dependent(cache8_merge_kernel<D>, dim3(grid.x * grid.y, kMergeSides), dim3(32 * kMergeWarps), 0, st, p);
}

template <int D>
cudaError_t cache8_nr(const Cache8Geom& g, const Cache8Args& a, void* ws, int* status, cudaStream_t st) {
  if (g.nr == 8) return cache8_d<D, 8>(g, a, ws, status, st);
  if constexpr (D <= 128) {
    if (g.nr == 32) return cache8_d<D, 32>(g, a, ws, status, st);
  }
  return cache8_d<D, 16>(g, a, ws, status, st);
}

}  // namespace

// Units (tiles of all segments) within 32 bits; 288 GB hold 18 million tiles, to be
// multiplied by up to 27 row blocks each.
bool cache8_fits(const Cache8Geom& g) {
  const double units = (double)g.B * g.Hkv * g.nmb * ((g.rows + T - 1) / T + g.visit);
  return units < 5.0e8 && (double)g.B * g.Hkv * g.M < 1.0e9;
}
// Query rows of a block.  Up to 8 rows need one group of softmax warps (the 48.8 us
// above are 57.9 with blocks of 16; D = 128, 43.9 and 46.0).  A tile costs blocks of 32
// nearly twice that of 16, and they read it once where two of 16 both do, one of them
// from L2.  At D = 256 and 512 the accumulators of 32 rows do not fit beside the scores
// of two CTAs.  At D <= 128 blocks of 32 are faster where CTAs have many tiles (32
// requests of 32 rows over 8,192 keys each, D = 128: 56.4 us, and 64.8 with 16; over up
// to 16,384, D = 64: 54.4 and 61.8).  With few the blocks of 16 spread better: 16
// requests, 2 kv heads, D = 64, 13.4 us, and 14.8 with 32, over up to 5,001 keys, of a
// cache with 4.2 tiles of 32 rows a CTA.  (The rule knows the cache's rows, not the
// lengths: 17.4 and 16.5 with 5,120 keys each.)
void cache8_split(Cache8Geom& g) {
  const long long units = (long long)g.B * g.Hkv * ((g.M + 31) / 32) * tiles_most(g);
  g.nr = g.M <= 8 ? 8 : g.M <= 16 || g.D > 128 || units < 6 * kCtas ? 16 : 32;
  g.nmb = (g.M + g.nr - 1) / g.nr;
  g.lanes = g.nmb < kCtas ? g.nmb : kCtas;
  // (in tiles; 0, 1, 2, 3 for all: 32 requests of 32 rows over up to 8,192 keys, D = 128, 43.2, 38.8, 37.5, 37.4 us; of
  // 16 rows 29.3, 26.6, 26.4, 26.5; 8 requests of 32 / 8 heads over up to 2,000 10.9, 9.4, 9.6, 9.7)
  g.visit = g.nr / 16 + 1;
}
size_t cache8_workspace_bytes(const Cache8Geom& g) { return c8_ws(g).total; }

cudaError_t launch_fwd_cache8(const Cache8Geom& g, const Cache8Args& a, void* ws, int* status, cudaStream_t st) {
  switch (g.D) {
    case 64: return cache8_nr<64>(g, a, ws, status, st);
    case 128: return cache8_nr<128>(g, a, ws, status, st);
    case 256: return cache8_nr<256>(g, a, ws, status, st);
    case 512: return cache8_nr<512>(g, a, ws, status, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace swa
