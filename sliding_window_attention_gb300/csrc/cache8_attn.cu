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
// Products are transposed: S^T (128 keys x 32) = K_tile [a b]^T and O^T (D x 48)
// += V_tile^T [hi mid lo]^T, so that the keys fill the MMA's M dimension whatever
// the number of query rows is.  One block has up to 16 rows (G * Lq of a kv head).
//
// Work.  The unit is one tile of 128 keys of one segment (request, kv head, row
// block).  The units of all requests, by the device-side lengths, are cut into
// 304 equal runs, one for each CTA, two CTAs an SM.  A segment that lies within
// one run is finished there; one that runs' ends cut leaves a partial (R, sum,
// O) for each run, and a second kernel merges those.
//
// Tiles are aligned to the end of what a request's rows see: one that would
// reach past it starts earlier (below key 0 the TMA fills zeros), so nothing
// behind a request's length is loaded.
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
constexpr int NR = 16;       // query rows of a block
constexpr int NS = 2 * NR;   // columns of S^T: q's two parts
constexpr int NP = 3 * NR;   // columns of O^T: a weight's three parts
constexpr int kCtas = 304;   // two an SM
constexpr int kThr = 224;    // TMA, MMA, four softmax warps, one that prepares queries
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
  int4* cuts;          // [kCtas]: segment of the CTA's first unit, the segment's units (begin, end), units in all
  float *ml, *po;      // partials [2 kCtas][rows of a block][2] and [..][D]
  int orow;            // rows of a partial's slot
  int* status;
};

// Key tiles of a request that any of its rows sees.
__device__ __forceinline__ int tiles_of(const Cache8Geom& g, int len) {
  const int n = min(len, g.rows);
  const int lo = g.W > 0 ? max(0, n - g.Lq - g.W + 1) : 0;
  return n > lo ? (n - lo + T - 1) / T : 0;
}

// The runs that the units are cut into, one for each CTA while they last; none is empty.
struct Runs {
  unsigned units, n;  // (units * kCtas < 2^32)
  __device__ __forceinline__ explicit Runs(unsigned u) : units(u), n(u < kCtas ? u : kCtas) {}
  __device__ __forceinline__ unsigned start(unsigned c) const { return c < n ? c * units / n : units; }
  __device__ __forceinline__ unsigned of(unsigned u) const { return ((u + 1) * n - 1) / units; }  // whose unit u is
};

// A place in a CTA's run: request, kv head, row block, tile.
struct Walk {
  const C8Params* p;
  int left;      // units from here to the end of the run
  int b, h, blk;
  int t, nt, n;  // tile of the segment, its tiles, the request's length
  bool first;    // first tile of this CTA's visit of the segment
  __device__ __forceinline__ void set_request() {
    n = min(p->kv_len[b], p->g.rows);
    nt = tiles_of(p->g, n);
  }
  __device__ __forceinline__ void begin(int b0, int r, int units) {  // unit r of request b0's
    b = b0;
    set_request();
    const int in = r / nt;
    t = r - in * nt;
    h = in / p->g.nmb;
    blk = in - h * p->g.nmb;
    left = units;
    first = true;
  }
  __device__ __forceinline__ int head() const { return b * p->g.Hkv + h; }
  __device__ __forceinline__ int key0() const { return n - T * (nt - t); }
  __device__ __forceinline__ bool last() const { return left == 1 || t == nt - 1; }
  __device__ __forceinline__ void next() {
    first = false;
    ++t;
    if (--left == 0 || t < nt) return;
    first = true;
    t = 0;
    if (++blk < p->g.nmb) return;
    blk = 0;
    if (++h < p->g.Hkv) return;
    h = 0;
    do {  // the next request with keys (there is one: units are left)
      ++b;
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

template <int D>
struct C8 {
  static constexpr int LINE = D < 128 ? D : 128;  // bytes of a key's line in a slot
  static constexpr int NCH = D / LINE;            // slots per tile and tensor; 128-row blocks of O^T
  static constexpr int SLOT = T * LINE;
  static constexpr int QB = NS * D;               // a block of queries: the parts' 32 rows
  static constexpr int PB = NP * T;               // weights
  // the softmax warps' small arrays: [2][4][16] exchanged maxima / sums, references, rescale factors, row
  // factors, row ranges, bounds and tags; the row factors of four visits
  static constexpr int RED = 0, REF = 512, ALPHA = REF + 64, FAC = ALPHA + 64, RNG = FAC + 64, BND = RNG + 128,
                       QFAC = BND + 64, SMALL = QFAC + 256;
  static constexpr int BARS = 256;
  static constexpr int FIT = (kSmemMax - 1024 - 2 * QB - PB - SMALL - BARS) / SLOT;
  static constexpr int NSLOT = FIT > 8 ? 8 : FIT;
  static constexpr int OFF_Q = NSLOT * SLOT, OFF_P = OFF_Q + 2 * QB, OFF_SMALL = OFF_P + PB, OFF_BAR = OFF_SMALL + SMALL;
  static constexpr size_t SMEM = (size_t)OFF_BAR + BARS + 1024;
  static constexpr uint32_t S_COL = 0, O_COL = 2 * NS;  // TMEM columns: S^T twice, O^T's blocks
  static constexpr uint32_t COLS = O_COL + NP * NCH;
  static constexpr uint32_t TCOLS = COLS <= 128 ? 128 : 256;  // (two CTAs share the 512)
  static_assert(COLS <= 256, "TMEM columns");
  static_assert(NSLOT >= 3 && SMEM <= (size_t)kSmemMax, "shared memory");
};

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
  __device__ __forceinline__ uint64_t* xch() const { return b + 24; }                 // the softmax warps' exchanges
  __device__ __forceinline__ uint64_t* drain() const { return b + 25; }
  static constexpr int kCount = 26;
  static __device__ __forceinline__ int arrivals(int i) { return i == 16 || i == 17 || i == 22 || i == 24 ? 4 : 1; }
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

// Column reduction of 16 columns over the warp's lanes by halving: lanes 2 c and 2 c + 1 end with column c in v[0].
template <bool MAX>
__device__ __forceinline__ void column_reduce(float (&v)[NR], int lane) {
  auto op = [](float a, float b) { return MAX ? fmaxf(a, b) : a + b; };
  int o = 16;
#pragma unroll
  for (int h = NR / 2; h >= 1; h >>= 1, o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < h; ++i) {
      const float give = up ? v[i] : v[i + h], keep = up ? v[i + h] : v[i];
      v[i] = op(keep, __shfl_xor_sync(0xffffffffu, give, o));
    }
  }
  v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], 1));
}

// Queries of one visit as the B operand of the first product: rows w, w + nw, ...
// of the block, the parts of row r in rows r and 16 + r, and each row's factor
// (what its scores are multiplied with, but for the keys' scales) in fac.
template <int D>
__device__ __forceinline__ void prepare_queries(const C8Params& p, int head, int blk, unsigned char* dst, float* fac,
                                                int w, int nw, int lane) {
  constexpr int E = D / 32;  // elements a lane
  const Cache8Geom& g = p.g;
  const uint16_t* src = p.q + ((size_t)head * g.M + blk * NR) * D + lane * E;
  const int rows = min(NR, g.M - blk * NR);
  const float sign = g.scale < 0.f ? -1.f : 1.f;
#pragma unroll 2
  for (int r = w; r < NR; r += nw) {
    float x[E];
    if (r < rows) {
      const uint16_t* s = src + (size_t)r * D;
      uint32_t v[E / 2];
      if constexpr (E == 2) v[0] = *reinterpret_cast<const uint32_t*>(s);
      else if constexpr (E == 4) *reinterpret_cast<uint2*>(v) = *reinterpret_cast<const uint2*>(s);
      else {
#pragma unroll
        for (int i = 0; i < E / 8; ++i) reinterpret_cast<uint4*>(v)[i] = reinterpret_cast<const uint4*>(s)[i];
      }
#pragma unroll
      for (int i = 0; i < E / 2; ++i) {
        x[2 * i] = __uint_as_float(v[i] << 16);
        x[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) x[i] = 0.f;
    }
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) amax = fmaxf(amax, fabsf(x[i]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const int e = cache8_scale_exponent(amax, -100);
    const float mul = sign * cache8_two_to(-e);
    uint16_t hi[E / 2], lo[E / 2];
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      const float a = x[2 * i] * mul, b = x[2 * i + 1] * mul;
      hi[i] = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
      const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(hi[i], __NV_E4M3);
      const float2 h = __half22float2(__half2(hr));
      lo[i] = __nv_cvt_float2_to_fp8x2(make_float2((a - h.x) * 16.f, (b - h.y) * 16.f), __NV_SATFINITE, __NV_E4M3);
    }
    // K-major rows in the swizzle of their line length
    const int col = lane * E, chunk = col / C8<D>::LINE, at = col % C8<D>::LINE;
    auto put = [&](int row, const uint16_t* v) {
      const int turn = D < 128 ? (row >> 1) & 3 : row & 7;
      unsigned char* d = dst + chunk * NS * C8<D>::LINE + row * C8<D>::LINE + (((at >> 4) ^ turn) << 4) + (at & 15);
      if constexpr (E == 2) *reinterpret_cast<uint16_t*>(d) = v[0];
      else if constexpr (E == 4) *reinterpret_cast<uint32_t*>(d) = v[0] | (uint32_t)v[1] << 16;
      else if constexpr (E == 8)
        *reinterpret_cast<uint2*>(d) = make_uint2(v[0] | (uint32_t)v[1] << 16, v[2] | (uint32_t)v[3] << 16);
      else
        *reinterpret_cast<uint4*>(d) = make_uint4(v[0] | (uint32_t)v[1] << 16, v[2] | (uint32_t)v[3] << 16,
                                                  v[4] | (uint32_t)v[5] << 16, v[6] | (uint32_t)v[7] << 16);
    };
    put(r, hi);
    put(NR + r, lo);
    if (lane == 0) fac[r] = fabsf(g.scale) * kLog2e * cache8_two_to(e);
  }
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

// The softmax warps' state over a run.
struct Soft {
  uint32_t at;   // TMEM: this thread's lane
  int n;         // tiles so far: S^T(n) is in buffer n & 1
  int xc;        // exchanges done
  int visit;
};

// One visit of a segment: its tiles' weights, then the result or the partial.
template <int D>
__device__ bool softmax_visit(const C8Params& p, unsigned char* base, const Bars& bar, volatile int* abort, Walk& w,
                              Soft& c) {
  using C = C8<D>;
  const Cache8Geom& g = p.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q4 = warp & 3, t = 32 * q4 + lane;
  unsigned char* small = base + C::OFF_SMALL;
  float* red = reinterpret_cast<float*>(small + C::RED);
  float* ref = reinterpret_cast<float*>(small + C::REF);
  float* alp = reinterpret_cast<float*>(small + C::ALPHA);
  float* fac = reinterpret_cast<float*>(small + C::FAC);
  int2* rng = reinterpret_cast<int2*>(small + C::RNG);
  int* bnd = reinterpret_cast<int*>(small + C::BND);
  volatile int* grow_tag = bnd + 8;    // [2] tile (plus one) at which some weight passed the top
  volatile int* scale_tag = bnd + 10;  // [1] tile (plus one) at which some row with earlier keys did
  const int blk = w.blk, head = w.head(), rows = min(NR, g.M - blk * NR);
  auto exchange = [&]() -> bool {  // what was written to shared memory before is visible after
    __syncwarp();
    if (lane == 0) mbar_arrive(bar.xch());
    const bool ok = wait(bar.xch(), c.xc & 1, abort);
    ++c.xc;
    return __all_sync(0xffffffffu, ok);
  };

  // the visit's first scores say that its queries' factors have been written
  if (!__all_sync(0xffffffffu, wait(bar.s_full(c.n & 1), (c.n >> 1) & 1, abort))) return false;
  // the visit is of the whole segment; row t's visible keys, and bounds over all rows
  const bool whole = w.t == 0 && w.left >= w.nt;
  {
    int lo = 0, hi = INT32_MAX;  // rows that are no query mask nothing: their columns are never read
    const bool row = t < rows;
    if (row) {
      hi = w.n - g.Lq + (blk * NR + t) % g.Lq;
      lo = g.W > 0 ? max(0, hi - g.W + 1) : 0;
    }
    if (t < NR) {
      rng[t] = make_int2(lo, hi);
      ref[t] = kUnset;
      fac[t] = reinterpret_cast<const float*>(small + C::QFAC)[(c.visit & 3) * NR + t];
    }
    const int lo_w = __reduce_max_sync(0xffffffffu, lo);
    const int hi_w = __reduce_min_sync(0xffffffffu, hi);
    if (lane == 0 && q4 == 0) {
      bnd[0] = lo_w;
      bnd[1] = hi_w;
    }
  }
  if (!exchange()) return false;
  const int lo_all = bnd[0], hi_all = bnd[1];  // (the rows are all in the first warp)

  float l_part[NR], m_row = kUnset;  // thread t < 16 holds row t's reference
#pragma unroll
  for (int q = 0; q < NR; ++q) l_part[q] = 0.f;
  const float* ks = p.ks + (size_t)head * g.nblk;
  const float* vs = p.vs + (size_t)head * g.nblk;
  const int at0 = max(w.key0() + t, 0) >> g.lb;
  float k_next = ks[at0], v_next = vs[at0];

  bool more = true, fresh = true;
#pragma unroll 1
  while (more) {
    const int n = c.n, buf = n & 1, key0 = w.key0();
    more = !w.last();
    const float kscale = k_next, vscale = fmaxf(v_next, cache8_two_to(kCache8LeastExponent));
    if (more) {  // the next tile's scales are under way meanwhile
      const int a = max(key0 + T + t, 0) >> g.lb;
      k_next = ks[a];
      v_next = vs[a];
    }
    const float lv = __log2f(vscale), iv = __frcp_rn(vscale);
    if (!__all_sync(0xffffffffu, wait(bar.s_full(buf), (n >> 1) & 1, abort))) return false;
    tc_fence_after();
    uint32_t sr[NS];
    tmem_ld32(c.at + C::S_COL + NS * buf, sr);
    tmem_wait_ld();
    float y[NR];
#pragma unroll
    for (int q = 0; q < NR; q += 4) {
      const float4 f = *reinterpret_cast<const float4*>(fac + q);
      const float ff[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        y[q + i] = fmaf(fmaf(__uint_as_float(sr[NR + q + i]), 0.0625f, __uint_as_float(sr[q + i])), ff[i] * kscale, lv);
    }
    if (!(key0 >= lo_all && key0 + T - 1 <= hi_all)) {
      const int key = key0 + t;
#pragma unroll
      for (int q = 0; q < NR; ++q) {
        const int2 r = rng[q];
        if (key < r.x || key > r.y) y[q] = -INFINITY;
      }
    }
    bool grow = fresh, scale = false;
    if (!fresh) {
      float over = -INFINITY;
#pragma unroll
      for (int q = 0; q < NR; q += 4) {
        const float4 f = *reinterpret_cast<const float4*>(ref + q);
        over = fmax3(over, y[q] - f.x, y[q + 1] - f.y);
        over = fmax3(over, y[q + 2] - f.z, y[q + 3] - f.w);
      }
      if (__any_sync(0xffffffffu, over > kTop) && lane == 0) grow_tag[n & 1] = n + 1;
      if (!exchange()) return false;
      grow = grow_tag[n & 1] == n + 1;
    }
    if (grow) {
      float* rb = red + (c.xc & 1) * 4 * NR;
      float mx[NR];
#pragma unroll
      for (int q = 0; q < NR; ++q) mx[q] = y[q];
      column_reduce<true>(mx, lane);
      if ((lane & 1) == 0) rb[q4 * NR + (lane >> 1)] = mx[0];
      if (!exchange()) return false;
      if (t < NR) {
        const float tm = fmaxf(fmaxf(rb[t], rb[NR + t]), fmaxf(rb[2 * NR + t], rb[3 * NR + t]));
        float a = 1.f;
        if (tm - m_row > kTop) {  // (a row without a key yet: its reference is the lowest number)
          const float to = tm - kBelow;
          if (m_row != kUnset) {
            a = fast_exp2(m_row - to);
            *scale_tag = n + 1;
          }
          m_row = to;
          ref[t] = to;
        }
        alp[t] = a;
      }
      if (!exchange()) return false;
      scale = *scale_tag == n + 1;
      if (scale) {
#pragma unroll
        for (int q = 0; q < NR; q += 4) {
          const float4 v = *reinterpret_cast<const float4*>(alp + q);
          l_part[q] *= v.x;
          l_part[q + 1] *= v.y;
          l_part[q + 2] *= v.z;
          l_part[q + 3] *= v.w;
        }
      }
    }
    fresh = false;
    // the weights 2^(y - reference), their row sums, and their three parts: hi is
    // a weight in fp16 rounded to its top byte, mid the rest so, lo the rest of that
    uint32_t part[3][NR / 4];
#pragma unroll
    for (int q = 0; q < NR; q += 4) {
      const float4 f = *reinterpret_cast<const float4*>(ref + q);
      const float e0 = fast_exp2(y[q] - f.x), e1 = fast_exp2(y[q + 1] - f.y);
      const float e2 = fast_exp2(y[q + 2] - f.z), e3 = fast_exp2(y[q + 3] - f.w);
      l_part[q] = fmaf(e0, iv, l_part[q]);
      l_part[q + 1] = fmaf(e1, iv, l_part[q + 1]);
      l_part[q + 2] = fmaf(e2, iv, l_part[q + 2]);
      l_part[q + 3] = fmaf(e3, iv, l_part[q + 3]);
      uint32_t a = pack_half2(e0, e1), b = pack_half2(e2, e3);
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        const uint32_t ra = a + 0x00800080u, rb = b + 0x00800080u;
        part[i][q / 4] = __byte_perm(ra, rb, 0x7531);
        if (i < 2) {
          const uint32_t ta = ra & 0xFF00FF00u, tb = rb & 0xFF00FF00u;
          const __half2 da = __hsub2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<const __half2*>(&ta));
          const __half2 db = __hsub2(*reinterpret_cast<__half2*>(&b), *reinterpret_cast<const __half2*>(&tb));
          a = *reinterpret_cast<const uint32_t*>(&da);
          b = *reinterpret_cast<const uint32_t*>(&db);
        }
      }
    }
    // the second product of tile n - 1 has finished with the weights' buffer, and with O^T before it is rescaled
    if (n > 0 && !__all_sync(0xffffffffu, wait(bar.o_done(), (n - 1) & 1, abort))) return false;
    if (scale) {  // uniform over the warps
      tc_fence_after();
#pragma unroll 1
      for (int i = 0; i < 3 * C::NCH; ++i) {
        uint32_t ov[NR];
        tmem_ld16(c.at + C::O_COL + NR * i, ov);
        tmem_wait_ld();
#pragma unroll
        for (int q = 0; q < NR; ++q) ov[q] = __float_as_uint(__uint_as_float(ov[q]) * alp[q]);
        tmem_st16(c.at + C::O_COL + NR * i, ov);
      }
      tmem_wait_st();
    }
    // MN-major operand without swizzle: a key's 16 rows of one part are 16 bytes
    unsigned char* pb = base + C::OFF_P + t * NR;
#pragma unroll
    for (int i = 0; i < 3; ++i)
      *reinterpret_cast<uint4*>(pb + i * T * NR) = make_uint4(part[i][0], part[i][1], part[i][2], part[i][3]);
    fence_proxy_async_smem();  // generic writes -> the tensor core's reads
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar.p_full());
    ++c.n;
    w.next();
  }
  ++c.visit;

  // row sums over the 128 threads, then O^T
  float* rb = red + (c.xc & 1) * 4 * NR;
  column_reduce<false>(l_part, lane);
  if ((lane & 1) == 0) rb[q4 * NR + (lane >> 1)] = l_part[0];
  if (!exchange()) return false;
  float* mul = alp;  // a whole segment's 1 / sum
  const size_t slot = (size_t)(2 * blockIdx.x + (c.visit > 1 ? 1 : 0)) * p.orow;
  if (t < rows) {
    const float l = (rb[t] + rb[NR + t]) + (rb[2 * NR + t] + rb[3 * NR + t]);
    if (whole) {
      const int m = blk * NR + t;
      float lse;
      mul[t] = finish_row(p.sinks ? p.sinks + (head % g.Hkv) * g.G + m / g.Lq : nullptr, m_row, l, &lse);
      p.lse[(size_t)head * g.M + m] = lse;
    } else {
      *reinterpret_cast<float2*>(p.ml + 2 * (slot + t)) = make_float2(m_row, l);
    }
  }
  if (whole && !exchange()) return false;
  if (!__all_sync(0xffffffffu, wait(bar.o_done(), (c.n - 1) & 1, abort))) return false;
  tc_fence_after();
#pragma unroll 1
  for (int h = 0; h < C::NCH; ++h) {
    uint32_t hi[NR], mid[NR], lo[NR];
    const uint32_t at = c.at + C::O_COL + NP * h;
    tmem_ld16(at, hi);  // warp-collective
    tmem_ld16(at + NR, mid);
    tmem_ld16(at + 2 * NR, lo);
    tmem_wait_ld();
    const int d = T * h + t;
    if (d < D) {
#pragma unroll
      for (int q = 0; q < NR; ++q)
        if (q < rows) {
          const float v = __uint_as_float(hi[q]) + (__uint_as_float(mid[q]) + __uint_as_float(lo[q]));
          if (whole)
            p.o[((size_t)head * g.M + blk * NR + q) * D + d] = __bfloat16_as_ushort(__float2bfloat16_rn(v * mul[q]));
          else p.po[(slot + q) * D + d] = v;
        }
    }
  }
  tc_fence_before();  // ordered before the next visit's first product by its arrival
  return true;
}

template <int D>
__global__ void __launch_bounds__(kThr, 2)
    cache8_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                  const __grid_constant__ C8Params p) {
  using C = C8<D>;
  constexpr int NW = kThr / 32, NSLOT = C::NSLOT, NCH = C::NCH;
  extern __shared__ unsigned char smem_raw[];
  __shared__ int scan_sum[NW], start_b, start_r;
  unsigned char* base = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const Bars bar{reinterpret_cast<uint64_t*>(base + C::OFF_BAR)};
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar.b + 30);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bar.b + 31);
  const Cache8Geom& g = p.g;
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, cta = blockIdx.x;

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  if (threadIdx.x < Bars::kCount) {
    mbar_init(bar.b + threadIdx.x, Bars::arrivals(threadIdx.x));
    fence_mbar_init();
  }
  if (threadIdx.x >= 32 && threadIdx.x < 36)  // the tags
    reinterpret_cast<int*>(base + C::OFF_SMALL + C::BND)[8 + threadIdx.x - 32] = 0;
  grid_dependency_wait();
  // Tensor memory is taken after the predecessor's end and before a dependent
  // may be placed: a grid that held columns while it waits for another that has
  // yet to allocate its own, on the same SM, would wait for ever.
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::TCOLS);
    tmem_relinquish();
  }
  // ---- the lengths: tiles in all
  const int nt0 = threadIdx.x < g.B ? tiles_of(g, p.kv_len[threadIdx.x]) : 0;  // of request threadIdx.x
  {
    int sum = nt0;
#pragma unroll 1
    for (int b = kThr + threadIdx.x; b < g.B; b += kThr) sum += tiles_of(g, p.kv_len[b]);
    sum = __reduce_add_sync(0xffffffffu, sum);
    if (lane == 0) scan_sum[warp] = sum;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_launch_dependents();  // the merge waits for this grid's end
  const uint32_t tmem = *tmem_slot;
  int tiles = 0;
#pragma unroll
  for (int i = 0; i < NW; ++i) tiles += scan_sum[i];
  const unsigned hn = g.Hkv * g.nmb;
  const Runs runs(tiles * hn);
  const unsigned u0 = runs.start(cta), u1 = runs.start(cta + 1);
  // ---- the request that unit u0 belongs to
  if (u0 < u1) {
    int before = 0;
#pragma unroll 1
    for (int c0 = 0; c0 < g.B; c0 += kThr) {
      const int b = c0 + threadIdx.x;
      const int nt = c0 == 0 ? nt0 : (b < g.B ? tiles_of(g, p.kv_len[b]) : 0);
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
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        const int v = scan_sum[i];
        if (i < warp) off += v;
        before += v;
      }
      if (nt > 0 && u0 >= off * hn && u0 < (off + nt) * hn) {
        start_b = b;
        start_r = (int)(u0 - off * hn);
      }
    }
    __syncthreads();
  }
  const int total = (int)(u1 - u0);
  auto walk = [&]() {
    Walk w;
    w.p = &p;
    w.begin(start_b, start_r, total);
    return w;
  };
  if (threadIdx.x == 0) {  // for the merge
    int4 cut = make_int4(-1, 0, 0, (int)runs.units);
    if (total > 0) {
      const Walk w = walk();
      const int begin = (int)u0 - w.t;
      cut = make_int4(w.head() * g.nmb + w.blk, begin, begin + w.nt, (int)runs.units);
    }
    p.cuts[cta] = cut;
  }

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (total > 0 && elect_one()) {
      // the cache, which a call reads once (but for further row blocks), gives way in L2
      const uint64_t policy = l2_policy(true);
      Walk wk = walk(), wv = wk;
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
      for (int n = -2; ok && n < total; ++n) ok = (n < 0 || load_tile(wv, &tmV)) && (n + 2 >= total || load_tile(wk, &tmK));
      if (*abort_flag) drain_ring(bar.slot_full(0), NSLOT, issued);  // loads in flight land before shared memory is released
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (total > 0 && elect_one()) {
      constexpr uint32_t idS = idesc_f8(T, NS, 0, 0, 0, 0);  // K x Q^T, both K-major, e4m3
      constexpr uint32_t idO = idesc_f8(T, NP, 0, 1, 1, 1);  // V^T (e4m3) x weights^T (e5m2), both MN-major
      constexpr uint32_t SWZ = D < 128 ? 4 : 2;
      // 8 lines make a swizzled group.  At D = 64 the second product's rows 64-127 repeat 0-63 and are never read.
      const uint64_t kd0 = smem_desc(smem_u32(base), D < 128 ? 0 : 16, 8 * C::LINE, SWZ);
      const uint64_t qd0 = smem_desc(smem_u32(base + C::OFF_Q), 16, 8 * C::LINE, SWZ);
      const uint64_t pd = smem_desc(smem_u32(base + C::OFF_P), 8 * NR, T * NR, 0);
      Walk ws = walk(), wv = ws;
      int used = 0, nq = 0;
      auto issue_s = [&](int n) -> bool {  // S^T(n) into buffer n & 1
        const int qs = nq & 1;
        if (ws.first && !wait(bar.q_full(qs), (nq >> 1) & 1, abort_flag)) return false;
#pragma unroll 1
        for (int c = 0; c < NCH; ++c, ++used) {
          const int s = used % NSLOT;
          if (!wait(bar.slot_full(s), (used / NSLOT) & 1, abort_flag)) return false;
          tc_fence_after();
          const uint64_t kd = desc_add(kd0, s * C::SLOT), qd = desc_add(qd0, qs * C::QB + c * NS * C::LINE);
#pragma unroll
          for (int k = 0; k < C::LINE / 32; ++k)
            mma_f8(tmem + C::S_COL + NS * (n & 1), desc_add(kd, k * 32), desc_add(qd, k * 32), idS, (c | k) ? 1u : 0u);
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
      for (int n = -2; ok && n < total; ++n) {
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
              mma_f8(tmem + C::O_COL + NP * c, desc_add(vd, k * 32 * C::LINE), desc_add(pd, k * 32 * NR), idO,
                     (acc || k > 0) ? 1u : 0u);
            mma_commit(bar.slot_empty(s));
          }
          if (!ok) break;
          mma_commit(bar.o_done());
          wv.next();
        }
        if (n + 2 < total) ok = issue_s(n + 2);  // after the second product of tile n: S buffer n & 1 is free
      }
      mma_commit(bar.drain());
      mbar_wait_drain(bar.drain(), 0);
    }
  } else if (warp < 6) {
    // ------------------------------------------------------------ softmax
    if (total > 0) {
      Walk w = walk();
      prepare_queries<D>(p, w.head(), w.blk, base + C::OFF_Q, reinterpret_cast<float*>(base + C::OFF_SMALL + C::QFAC),
                         warp - 2, 4, lane);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar.q_full(0));
      bool ok = true;
      Soft c{tmem + ((uint32_t)(32 * (warp & 3)) << 16), 0, 0, 0};
#pragma unroll 1
      while (ok && w.left > 0) ok = softmax_visit<D>(p, base, bar, abort_flag, w, c);
    }
  } else {
    // ------------------------------------------------------------ the later visits' queries
    if (total > 0) {
      Walk w = walk();
      w.skip();
#pragma unroll 1
      for (int v = 1; w.left > 0; ++v) {
        const int s = v & 1;
        if (v >= 2 && !__all_sync(0xffffffffu, wait(bar.q_empty(s), ((v >> 1) & 1) ^ 1, abort_flag))) break;
        prepare_queries<D>(p, w.head(), w.blk, base + C::OFF_Q + s * C::QB,
                           reinterpret_cast<float*>(base + C::OFF_SMALL + C::QFAC) + (v & 3) * NR, 0, 1, lane);
        __syncwarp();
        if (lane < 4) mbar_arrive(bar.q_full(s));
        w.skip();
      }
    }
    // requests without a key: no unit is theirs
#pragma unroll 1
    for (int b = cta; b < g.B; b += kCtas) {
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
    tmem_dealloc(tmem, C::TCOLS);
  }
}

// Merge of one row of the segment that the begin of run blockIdx.x cuts: the
// first cut of a segment does it for all of them.  With R = max R_i over the
// partials, o = sum 2^(R_i - R) O_i / sum 2^(R_i - R) l_i.
template <int D>
__global__ void __launch_bounds__(128) cache8_merge_kernel(const __grid_constant__ C8Params p) {
  constexpr int LANES = D / 4, GR = 128 / LANES, AHEAD = D == 512 ? 6 : 8;
  __shared__ float4 part[GR][LANES];
  const Cache8Geom& g = p.g;
  const int cta = blockIdx.x, row = blockIdx.y, lane = threadIdx.x & 31;
  grid_launch_dependents();
  grid_dependency_wait();
  const int4 cut = p.cuts[cta];
  if (cut.x < 0) return;
  const Runs runs(cut.w);
  const unsigned u0 = cut.y, u1 = cut.z;
  const int c0 = (int)runs.of(u0);
  if (c0 != cta - 1) return;  // the run begins with the segment (c0 == cta), or an earlier cut is the first
  const int head = cut.x / g.nmb, blk = cut.x - head * g.nmb, rows = min(NR, g.M - blk * NR);
  if (row >= rows) return;
  const int n = (int)runs.of(u1 - 1) - c0 + 1;
  const int slot0 = 2 * c0 + (runs.start(c0) == u0 ? 0 : 1);
  auto slot_of = [&](int i) { return (size_t)(i == 0 ? slot0 : 2 * (c0 + i)) * p.orow + row; };
  auto ml_of = [&](int i) { return *reinterpret_cast<const float2*>(p.ml + 2 * slot_of(i)); };
  const int grp = threadIdx.x / LANES, d = threadIdx.x % LANES;
  auto o_of = [&](int i) { return *reinterpret_cast<const float4*>(p.po + slot_of(i) * D + 4 * d); };
  // all first loads are under way before any is used
  const float2 first = lane < n ? ml_of(lane) : make_float2(kUnset, 0.f);
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
  float mx = first.x;
#pragma unroll 1
  for (int i = lane + 32; i < n; i += 32) mx = fmaxf(mx, ml_of(i).x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  // (a part without a visible key: its sum and O are 0)
  auto weight = [&](float x) { return exp2f(x - mx); };
  float l = weight(first.x) * first.y;
#pragma unroll 1
  for (int i = lane + 32; i < n; i += 32) {
    const float2 t = ml_of(i);
    l += weight(t.x) * t.y;
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
  const int m = blk * NR + row;
  float lse;
  const float inv = finish_row(p.sinks ? p.sinks + (head % g.Hkv) * g.G + m / g.Lq : nullptr, mx, l, &lse);
  const __nv_bfloat162 a = __floats2bfloat162_rn(acc.x * inv, acc.y * inv), b = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
  const size_t at = (size_t)head * g.M + m;
  *reinterpret_cast<uint2*>(p.o + at * D + 4 * d) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  if (d == 0) p.lse[at] = lse;
}

struct C8Ws {
  size_t cuts, ml, po, total;
};
int slot_rows(const Cache8Geom& g) { return g.M < NR ? g.M : NR; }
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

template <int D>
cudaError_t cache8_d(const Cache8Geom& g, const Cache8Args& a, void* ws, int* status, cudaStream_t st) {
  using C = C8<D>;
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
  auto kern = cache8_kernel<D>;
  static std::atomic<unsigned long long> done{0};
  if ((e = allow_smem(kern, (int)C::SMEM, done)) != cudaSuccess) return e;
  // both are programmatic dependents of what runs before them: the main grid's
  // set-up and the merge's placement fall into its predecessor's end
  if ((e = launch_dependent(kern, dim3(kCtas), dim3(kThr), C::SMEM, st, tk, tv, p)) != cudaSuccess) return e;
  return launch_dependent(cache8_merge_kernel<D>, dim3(kCtas, p.orow), dim3(128), 0, st, p);
}

}  // namespace

// Units (tiles of all segments) times runs within 32 bits.
bool cache8_fits(const Cache8Geom& g) {
  const double units = (double)g.B * g.Hkv * g.nmb * ((g.rows + T - 1) / T);
  return units * kCtas < 4.0e9 && (double)g.B * g.Hkv * g.M < 1.0e9;
}
int cache8_row_blocks(int M) { return (M + NR - 1) / NR; }
size_t cache8_workspace_bytes(const Cache8Geom& g) { return c8_ws(g).total; }

cudaError_t launch_fwd_cache8(const Cache8Geom& g, const Cache8Args& a, void* ws, int* status, cudaStream_t st) {
  switch (g.D) {
    case 64: return cache8_d<64>(g, a, ws, status, st);
    case 128: return cache8_d<128>(g, a, ws, status, st);
    case 256: return cache8_d<256>(g, a, ws, status, st);
    case 512: return cache8_d<512>(g, a, ws, status, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace swa
