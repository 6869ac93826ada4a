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
// the product of one block of query rows with one kv head's prefix (up to NP
// rows, packed from as many requests as fit, so the prefix is read once for
// all of them), or with one request's own cache (up to 16 rows: the G * Lq
// rows of a kv head).  One CTA per SM takes an equal run of units, however
// ragged the lengths: every CTA sums the device-side lengths itself, no host
// sees them and no counter has to be reset between calls.  A CTA's share of a
// segment leaves one partial (m, l, O) in the slot cta + segment, which no
// other pair of them has; a second kernel merges a row's partials.
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

constexpr int kThr = 192;   // warp 0 TMA, warp 1 MMA, warps 2-5 softmax (thread = key = TMEM lane)
constexpr int T = 128;      // keys per tile
constexpr int kOwnRows = 16;  // query rows of an own segment (MMA N)
constexpr int kSMs = 152;   // one CTA per SM
constexpr int kSmemMax = 232448;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleLog2 = 8.0f;
constexpr int kPlanInts = 4;  // plan words in front of the per-request offsets

struct SharedParams {
  SharedGeom g;
  SharedSplit s;
  const int* own_len;
  const float* sinks;  // [Hq] or null
  uint16_t* o;         // bf16 [B, Hq, Lq, D]
  float* lse;          // [B, Hq, Lq]
  int* plan;           // {prefix tiles, units, CTAs with work, prefix start}, then own tiles before each request
  float *pp_ml, *pp_o;  // prefix partials: [slot][rows][2] and [slot][rows][D]
  float *po_ml, *po_o;  // own partials
  int* status;
};

// First own key any of a request's rows sees, and the tiles from there to
// the end of its cache; a negative length is an empty place of the batch.
__device__ __forceinline__ int own_tiles(const SharedGeom& g, int len) {
  const int n = min(len, g.own_rows);
  const int lo = g.W > 0 ? max(0, n - g.Lq - g.W + 1) : 0;
  return n > lo ? (n - lo + T - 1) / T : 0;
}

// A place in a CTA's run of units.
struct Walk {
  const SharedParams* p;
  int left;        // units from here to the end of the run (0: done)
  int own;         // this segment: a request's own cache, or the prefix
  int seg;         // index among the segments of its kind
  int h, b, blk;   // kv head; request (own); row block
  int t, nt, n;    // tile of the segment, its tiles, own length
  int key_lo;      // prefix: first key of tile 0
  bool first;      // first tile of this CTA's visit of the segment

  __device__ __forceinline__ void set_own() {
    n = min(p->own_len[b], p->g.own_rows);
    nt = own_tiles(p->g, n);
  }
  __device__ __forceinline__ int key0() const { return own ? n - T * (nt - t) : key_lo + T * t; }
  __device__ __forceinline__ bool last() const { return left == 1 || t == nt - 1; }
  __device__ __forceinline__ void next() {
    first = false;
    ++t;
    if (--left == 0 || t < nt) return;
    first = true;
    t = 0;
    if (!own) {
      ++seg;
      if (++blk == p->s.nrb) {
        blk = 0;
        ++h;
      }
      if (h < p->g.Hkv) return;
      own = 1;
      h = 0;
      b = -1;
    } else {
      if (++blk < p->s.nomb) {
        ++seg;
        return;
      }
      blk = 0;
      if (++h < p->g.Hkv) {
        ++seg;
        return;
      }
      h = 0;
    }
    do {  // the next request with keys (there is one: units are left)
      ++b;
      set_own();
    } while (nt == 0);
    seg = b * p->g.Hkv * p->s.nomb;
  }
};

template <int D, int NP>
struct ShCfg {
  static constexpr int NCH = D / 64;             // 64-column chunks of a row
  static constexpr int CPS = NCH < 2 ? NCH : 2;  // chunks per ring slot
  static constexpr int SPT = NCH / CPS;          // slots per tile and tensor
  static constexpr int NDC = (D + 127) / 128;    // 128-column blocks of O^T
  static constexpr int SLOT = CPS * T * 128;
  static constexpr int QP = NP * D * 2, QO = kOwnRows * D * 2;
  static constexpr int QD = (D == 512 && NP > 16) ? 1 : 2;  // buffers of own queries
  static constexpr int PB = NP > 16 ? NP * T * 2 : kOwnRows * T * 2;  // one P^T buffer
  // behind the ring: prefix queries, own queries, P^T, then the small arrays
  static constexpr int SMALL = 2 * 4 * NP * 4 + 3 * NP * 4 + NP * 8 + 64 + 512;
  // at head dim 64 the second product's 128 rows read one chunk past a slot
  // (rows 64-127 of O^T, never used): the last slot's must stay in bounds
  static constexpr int TAIL = D == 64 ? T * 128 : 0;
  static constexpr int FIXED = QP + QD * QO + 2 * PB + SMALL + TAIL;
  static constexpr int FIT = (kSmemMax - 1024 - FIXED) / SLOT;
  static constexpr int NSLOT = FIT > 8 ? 8 : FIT;
  static constexpr int OFF_QP = NSLOT * SLOT;
  static constexpr int OFF_QO = OFF_QP + QP;
  static constexpr int OFF_P = OFF_QO + QD * QO;
  static constexpr int OFF_RED = OFF_P + 2 * PB;       // [2][4 warps][NP] exchanged maxima / sums
  static constexpr int OFF_THR = OFF_RED + 2 * 4 * NP * 4;  // [NP] reference maximum + kRescaleLog2
  static constexpr int OFF_USE = OFF_THR + NP * 4;     // [NP] reference maximum (0 where there is none)
  static constexpr int OFF_ALPHA = OFF_USE + NP * 4;   // [NP] rescale factors
  static constexpr int OFF_RNG = OFF_ALPHA + NP * 4;   // [NP] visible keys (first, last) of each row
  static constexpr int OFF_BND = OFF_RNG + NP * 8;     // [4][2] bounds over a warp's rows, [2] growth tags
  static constexpr int OFF_BAR = OFF_BND + 64;
  static constexpr size_t SMEM = (size_t)OFF_BAR + 512 + TAIL + 1024;
  static constexpr uint32_t S_COL = 0, O_COL = 2 * NP;  // TMEM columns
  static constexpr uint32_t TCOLS = O_COL + NDC * NP <= 128 ? 128 : (O_COL + NDC * NP <= 256 ? 256 : 512);
  static_assert(NSLOT >= 2 && SMEM + 256 <= (size_t)kSmemMax, "shared memory");
  static_assert(O_COL + NDC * NP <= 512, "TMEM columns");
  static_assert(NP == 16 || NP == 64, "row block");
};

// Column reduction over the warp's 32 lanes by halving: each step keeps one
// half of the columns and hands the other half over, so N columns take N
// shuffles (5 N for a butterfly a column).  N = 64: lane l ends with columns
// 2 l, 2 l + 1 in v[0], v[1]; N = 16: lanes 2 c, 2 c + 1 with column c in v[0].
template <int N, bool MAX>
__device__ __forceinline__ void column_reduce(float (&v)[N], int lane) {
  auto op = [](float a, float b) { return MAX ? fmaxf(a, b) : a + b; };
  int o = 16;
#pragma unroll
  for (int h = N / 2; h >= (N == 64 ? 2 : 1); h >>= 1, o >>= 1) {
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
  if (N == 64) *reinterpret_cast<float2*>(dst + 2 * lane) = make_float2(v[0], v[1]);
  else if ((lane & 1) == 0) dst[lane >> 1] = v[0];
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// What the softmax warps share.
struct SoftCtx {
  unsigned char* base;
  uint64_t *s_full, *p_full, *o_done, *xch;
  volatile int* abort;
  uint32_t tmem;
  int n;   // tiles done by this CTA
  int xc;  // exchanges done
};

// Every softmax thread arrives and waits (bounded); what was written to
// shared memory before is visible after.
__device__ __forceinline__ bool exchange(SoftCtx& c) {
  mbar_arrive(c.xch);
  const bool ok = mbar_wait(c.xch, c.xc & 1, c.abort);
  ++c.xc;
  return __all_sync(0xffffffffu, ok);
}

// One visit of a segment: its tiles' softmax, then the partial result.
// N = 16: every thread keeps all rows' running maxima in registers, and each
// tile exchanges its column maxima.  N = 64: the maxima live in shared memory,
// and a tile exchanges only whether any score outgrew its row's reference by
// more than 2^kRescaleLog2 (rare after a visit's first tiles).
template <int D, int NP, int N>
__device__ bool softmax_visit(const SharedParams& p, Walk& w, SoftCtx& c) {
  using C = ShCfg<D, NP>;
  constexpr int NDC = C::NDC;
  const SharedGeom& g = p.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q4 = warp & 3, t = 32 * q4 + lane;
  const uint32_t lane_off = (uint32_t)(32 * q4) << 16;
  const float sl2 = g.scale * kLog2e;
  float* red = reinterpret_cast<float*>(c.base + C::OFF_RED);
  float* thr = reinterpret_cast<float*>(c.base + C::OFF_THR);
  float* use = reinterpret_cast<float*>(c.base + C::OFF_USE);
  float* alp = reinterpret_cast<float*>(c.base + C::OFF_ALPHA);
  int2* rng = reinterpret_cast<int2*>(c.base + C::OFF_RNG);
  int* bnd = reinterpret_cast<int*>(c.base + C::OFF_BND);
  volatile int* grow_tag = bnd + 8;
  const Walk at = w;  // this visit

  // visible keys of row t (own cache: own indices), and bounds over all rows
  {
    int lo = 0, hi = INT32_MAX;  // rows that are no query mask nothing: their columns are never read
    bool row = false;
    if (t < N) {
      if (at.own) {
        const int m = at.blk * kOwnRows + t, i = m % g.Lq;
        row = m < g.M;
        if (row) {
          hi = at.n - g.Lq + i;
          lo = g.W > 0 ? max(0, hi - g.W + 1) : 0;
        }
      } else {
        const int b = at.blk / p.s.nmb * p.s.nb + t / p.s.mb, m = at.blk % p.s.nmb * NP + t % p.s.mb;
        const int len = (t < p.s.prow && b < g.B && m < g.M) ? p.own_len[b] : -1;
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

  float l_part[N], m_run[N == 16 ? 16 : 1];  // N = 64: thread t holds row t's reference maximum
#pragma unroll
  for (int q = 0; q < N; ++q) l_part[q] = 0.f;
  if constexpr (N == 16) {
#pragma unroll
    for (int q = 0; q < N; ++q) m_run[q] = -INFINITY;
  } else {
    m_run[0] = -INFINITY;
  }

  bool more = true;
  while (more) {
    const int n = c.n, key0 = w.key0();
    const bool first = w.first;
    more = !w.last();
    if (!__all_sync(0xffffffffu, mbar_wait(c.s_full + (n & 1), (n >> 1) & 1, c.abort))) return false;
    tc_fence_after();
    uint32_t sr[N];
    if constexpr (N == 16) {
      tmem_ld16(c.tmem + lane_off + C::S_COL + NP * (n & 1), sr);
    } else {
      tmem_ld32(c.tmem + lane_off + C::S_COL + NP * (n & 1), *reinterpret_cast<uint32_t(*)[32]>(sr));
      tmem_ld32(c.tmem + lane_off + C::S_COL + NP * (n & 1) + 32, *reinterpret_cast<uint32_t(*)[32]>(sr + 32));
    }
    tmem_wait_ld();
    float x[N];
    if (key0 >= lo_all && key0 + T - 1 <= hi_all) {
#pragma unroll
      for (int q = 0; q < N; ++q) x[q] = __uint_as_float(sr[q]) * sl2;
    } else {
      const int key = key0 + t;
#pragma unroll
      for (int q = 0; q < N; ++q) {
        const int2 r = rng[q];
        x[q] = (key >= r.x && key <= r.y) ? __uint_as_float(sr[q]) * sl2 : -INFINITY;
      }
    }
    bool waited = false;  // for PV(n - 1)
    if constexpr (N == 16) {
      float mx[N];
#pragma unroll
      for (int q = 0; q < N; ++q) mx[q] = x[q];
      column_reduce<N, true>(mx, lane);
      float* rb = red + (c.xc & 1) * 4 * NP;
      column_post<N>(mx, rb + q4 * NP, lane);
      if (!exchange(c)) return false;
      bool grow = false;
      float alpha[N];
#pragma unroll
      for (int q = 0; q < N; ++q) {
        const float tm = fmaxf(fmaxf(rb[q], rb[NP + q]), fmaxf(rb[2 * NP + q], rb[3 * NP + q]));
        alpha[q] = 1.f;
        if (tm > m_run[q] + kRescaleLog2) {  // the reference maximum moves (lazily)
          if (m_run[q] != -INFINITY) {
            alpha[q] = exp2f(m_run[q] - tm);
            grow = true;
          }
          m_run[q] = tm;
        }
      }
      if (grow) {  // uniform: every thread holds the same maxima
        if (n > 0 && !__all_sync(0xffffffffu, mbar_wait(c.o_done, (n - 1) & 1, c.abort))) return false;
        waited = true;
        tc_fence_after();
#pragma unroll
        for (int h = 0; h < NDC; ++h) {
          uint32_t ov[16];
          tmem_ld16(c.tmem + lane_off + C::O_COL + NP * h, ov);
          tmem_wait_ld();
#pragma unroll
          for (int q = 0; q < N; ++q) ov[q] = __float_as_uint(__uint_as_float(ov[q]) * alpha[q]);
          tmem_st16(c.tmem + lane_off + C::O_COL + NP * h, ov);
        }
        tmem_wait_st();
#pragma unroll
        for (int q = 0; q < N; ++q) l_part[q] *= alpha[q];
      }
#pragma unroll
      for (int q = 0; q < N; ++q) {
        x[q] = fast_exp2(x[q] - (m_run[q] == -INFINITY ? 0.f : m_run[q]));
        l_part[q] += x[q];
      }
    } else {
      bool grow = first;
      if (!first) {
        bool over = false;
#pragma unroll
        for (int q = 0; q < N; q += 4) {
          const float4 v = *reinterpret_cast<const float4*>(thr + q);
          over |= x[q] > v.x || x[q + 1] > v.y || x[q + 2] > v.z || x[q + 3] > v.w;
        }
        if (__any_sync(0xffffffffu, over) && lane == 0) grow_tag[n & 1] = n + 1;
        if (!exchange(c)) return false;
        grow = grow_tag[n & 1] == n + 1;
      }
      if (grow) {
        float mx[N];
#pragma unroll
        for (int q = 0; q < N; ++q) mx[q] = x[q];
        column_reduce<N, true>(mx, lane);
        float* rb = red + (c.xc & 1) * 4 * NP;
        column_post<N>(mx, rb + q4 * NP, lane);
        if (!exchange(c)) return false;
        if (t < N) {
          const float tm = fmaxf(fmaxf(rb[t], rb[NP + t]), fmaxf(rb[2 * NP + t], rb[3 * NP + t]));
          float a = 1.f;
          if (tm > m_run[0] + kRescaleLog2) {
            if (m_run[0] != -INFINITY) a = exp2f(m_run[0] - tm);
            m_run[0] = tm;
            use[t] = tm;
            thr[t] = tm + kRescaleLog2;
          } else if (first) {
            use[t] = 0.f;  // no visible key yet
          }
          alp[t] = a;
        }
        if (!exchange(c)) return false;
        if (!first) {
          if (!__all_sync(0xffffffffu, mbar_wait(c.o_done, (n - 1) & 1, c.abort))) return false;
          waited = true;
          tc_fence_after();
#pragma unroll 1
          for (int h = 0; h < NDC; ++h)
#pragma unroll
            for (int hf = 0; hf < N / 32; ++hf) {
              uint32_t ov[32];
              tmem_ld32(c.tmem + lane_off + C::O_COL + NP * h + 32 * hf, ov);
              tmem_wait_ld();
#pragma unroll
              for (int q = 0; q < 32; ++q) ov[q] = __float_as_uint(__uint_as_float(ov[q]) * alp[32 * hf + q]);
              tmem_st32(c.tmem + lane_off + C::O_COL + NP * h + 32 * hf, ov);
            }
          tmem_wait_st();
#pragma unroll
          for (int q = 0; q < N; ++q) l_part[q] *= alp[q];
        }
      }
#pragma unroll
      for (int q = 0; q < N; q += 4) {
        const float4 v = *reinterpret_cast<const float4*>(use + q);
        x[q] = fast_exp2(x[q] - v.x);
        x[q + 1] = fast_exp2(x[q + 1] - v.y);
        x[q + 2] = fast_exp2(x[q + 2] - v.z);
        x[q + 3] = fast_exp2(x[q + 3] - v.w);
#pragma unroll
        for (int e = 0; e < 4; ++e) l_part[q + e] += x[q + e];
      }
    }
    // PV(n - 1) has finished, so PV(n - 2), the last reader of P buffer n & 1, has too
    if (!waited && n > 0 && !__all_sync(0xffffffffu, mbar_wait(c.o_done, (n - 1) & 1, c.abort))) return false;
    unsigned char* pb = c.base + C::OFF_P + (n & 1) * C::PB;
    if constexpr (N == 16) {
      // K-major B operand: row q, key t -> chunk t / 64, 128-byte swizzle
      pb += (t >> 6) * kOwnRows * 128;
      const int kc = t & 63;
#pragma unroll
      for (int q = 0; q < N; ++q)
        *reinterpret_cast<__nv_bfloat16*>(pb + q * 128 + (((kc >> 3) ^ (q & 7)) << 4) + (kc & 7) * 2) =
            __float2bfloat16_rn(x[q]);
    } else {
      // MN-major B operand: key t's 64 rows are one 128-byte swizzled line
#pragma unroll
      for (int u = 0; u < 8; ++u)
        *reinterpret_cast<uint4*>(pb + t * 128 + ((u ^ (t & 7)) << 4)) =
            make_uint4(pack_bf16(x[8 * u], x[8 * u + 1]), pack_bf16(x[8 * u + 2], x[8 * u + 3]),
                       pack_bf16(x[8 * u + 4], x[8 * u + 5]), pack_bf16(x[8 * u + 6], x[8 * u + 7]));
    }
    fence_proxy_async_smem();  // generic writes -> the tensor core's reads
    tc_fence_before();
    mbar_arrive(c.p_full + (n & 1));
    ++c.n;
    w.next();
  }

  // the visit's partial: row sums over the 128 threads, then O^T
  column_reduce<N, false>(l_part, lane);
  float* rb = red + (c.xc & 1) * 4 * NP;
  column_post<N>(l_part, rb + q4 * NP, lane);
  if (!exchange(c)) return false;
  if (!__all_sync(0xffffffffu, mbar_wait(c.o_done, (c.n - 1) & 1, c.abort))) return false;
  tc_fence_after();
  const size_t slot = (size_t)blockIdx.x + at.seg;
  const int stride = at.own ? p.s.orow : p.s.prow;  // rows of a slot
  int rows;                                         // of which this segment has
  if (at.own) rows = min(kOwnRows, g.M - at.blk * kOwnRows);
  else if (p.s.nmb > 1) rows = min(NP, g.M - at.blk % p.s.nmb * NP);
  else rows = min(p.s.nb, g.B - at.blk * p.s.nb) * g.M;
  float* out = (at.own ? p.po_o : p.pp_o) + slot * stride * D;
  float* ml = (at.own ? p.po_ml : p.pp_ml) + slot * stride * 2;
  if (t < rows) {
    float m;
    if constexpr (N == 16) {
      m = m_run[0];
#pragma unroll
      for (int q = 1; q < N; ++q) m = t == q ? m_run[q] : m;
    } else {
      m = m_run[0];
    }
    *reinterpret_cast<float2*>(ml + 2 * t) =
        make_float2(m, (rb[t] + rb[NP + t]) + (rb[2 * NP + t] + rb[3 * NP + t]));
  }
#pragma unroll 1
  for (int h = 0; h < NDC; ++h) {
    const int d = 128 * h + t;
#pragma unroll
    for (int part = 0; part < N / 16; ++part) {
      uint32_t ov[16];
      tmem_ld16(c.tmem + lane_off + C::O_COL + NP * h + 16 * part, ov);  // warp-collective
      tmem_wait_ld();
      if (d < D) {
#pragma unroll
        for (int q = 0; q < 16; ++q)
          if (16 * part + q < rows) out[(size_t)(16 * part + q) * D + d] = __uint_as_float(ov[q]);
      }
    }
  }
  tc_fence_before();  // ordered before the next visit's first PV by its P arrival
  return true;
}

template <int D, int NP>
__global__ void __launch_bounds__(kThr, 1)
    shared_kernel(const __grid_constant__ CUtensorMap tmQP, const __grid_constant__ CUtensorMap tmQO,
                  const __grid_constant__ CUtensorMap tmKP, const __grid_constant__ CUtensorMap tmVP,
                  const __grid_constant__ CUtensorMap tmKO, const __grid_constant__ CUtensorMap tmVO,
                  const __grid_constant__ SharedParams p) {
  using C = ShCfg<D, NP>;
  constexpr int NCH = C::NCH, CPS = C::CPS, SPT = C::SPT, NSLOT = C::NSLOT, QD = C::QD;
  extern __shared__ unsigned char smem_raw[];
  __shared__ int scan_sum[6], scan_min[6], start_b, start_r;
  unsigned char* base = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(base + C::OFF_BAR);
  uint64_t* slot_full = bars;                  // [NSLOT]
  uint64_t* slot_empty = slot_full + NSLOT;    // [NSLOT]
  uint64_t* qp_full = slot_empty + NSLOT;      // [1] prefix queries of a visit
  uint64_t* qp_empty = qp_full + 1;            // [1]
  uint64_t* qo_full = qp_empty + 1;            // [QD] own queries
  uint64_t* qo_empty = qo_full + QD;           // [QD]
  uint64_t* s_full = qo_empty + QD;            // [2] S^T(n) in TMEM
  uint64_t* p_full = s_full + 2;               // [2] P^T(n) written (and O^T rescaled)
  uint64_t* o_done = p_full + 2;               // [1] PV(n) finished
  uint64_t* xch = o_done + 1;                  // [1] softmax threads' exchanges
  uint64_t* mma_drain = xch + 1;               // [1]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const SharedGeom& g = p.g;
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  grid_launch_dependents();  // the merge waits for this grid's end

  // ---- this CTA's run of units, from the lengths on the device
  {
    int sum = 0, mn = INT32_MAX;
    for (int b = threadIdx.x; b < g.B; b += kThr) {
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
  if (threadIdx.x == 0) start_b = -1;
  __syncthreads();
  int tiles = 0, mn = INT32_MAX;
#pragma unroll
  for (int i = 0; i < 6; ++i) {
    tiles += scan_sum[i];
    mn = min(mn, scan_min[i]);
  }
  // prefix keys that some row sees start at key_lo (none without a live request)
  const int key_lo = mn == INT32_MAX ? g.P : (g.W > 0 ? min(g.P, max(0, g.P + mn - g.Lq - g.W + 1)) : 0);
  const int tp = (g.P - key_lo + T - 1) / T;
  const int hn = g.Hkv * p.s.nomb;
  const int up = g.Hkv * p.s.nrb * tp, units = up + tiles * hn;
  const int ctas = min((int)gridDim.x, units);
  const int cta = blockIdx.x;
  if (cta == 0 && threadIdx.x == 0) {
    p.plan[0] = tp;
    p.plan[1] = units;
    p.plan[2] = ctas;
    p.plan[3] = key_lo;
  }
  if (cta >= ctas && cta != 0) return;
  const int u0 = ctas ? (int)((long long)units * cta / ctas) : 0;
  const int u1 = ctas ? (int)((long long)units * (cta + 1) / ctas) : 0;
  // the request that unit u0 belongs to (own units only); CTA 0 writes every
  // request's offset for the merge
  if (u0 >= up || cta == 0) {
    int before = 0;
    for (int c0 = 0; c0 < g.B; c0 += kThr) {
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
      for (int i = 0; i < 6; ++i) {
        if (i < warp) off += scan_sum[i];
        before += scan_sum[i];
      }
      if (cta == 0 && b < g.B) p.plan[kPlanInts + b] = off;
      const int v = u0 - up;
      if (nt > 0 && v >= off * hn && v < (off + nt) * hn) {
        start_b = b;
        start_r = v - off * hn;
      }
    }
  }
  if (ctas == 0) return;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NSLOT; ++s) {
      mbar_init(slot_full + s, 1);
      mbar_init(slot_empty + s, 1);
    }
    mbar_init(qp_full, 1);
    mbar_init(qp_empty, 1);
    for (int s = 0; s < QD; ++s) {
      mbar_init(qo_full + s, 1);
      mbar_init(qo_empty + s, 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(s_full + s, 1);
      mbar_init(p_full + s, 128);
    }
    mbar_init(o_done, 1);
    mbar_init(xch, 128);
    mbar_init(mma_drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  // rows of the prefix query block that no box fills stay zero
  for (int i = threadIdx.x; i < C::QP / 16; i += kThr) reinterpret_cast<uint4*>(base + C::OFF_QP)[i] = make_uint4(0, 0, 0, 0);
  if (threadIdx.x < 2) reinterpret_cast<int*>(base + C::OFF_BND)[8 + threadIdx.x] = 0;  // growth tags
  fence_proxy_async_smem();
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::TCOLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  Walk w0;
  w0.p = &p;
  w0.left = u1 - u0;
  w0.key_lo = key_lo;
  w0.first = true;
  w0.n = 0;
  if (u0 < up) {
    w0.own = 0;
    w0.seg = u0 / tp;
    w0.t = u0 - w0.seg * tp;
    w0.nt = tp;
    w0.h = w0.seg / p.s.nrb;
    w0.blk = w0.seg - w0.h * p.s.nrb;
    w0.b = 0;
  } else {
    w0.own = 1;
    w0.b = start_b;
    w0.set_own();
    const int in = start_r / w0.nt;  // (kv head, row block)
    w0.t = start_r - in * w0.nt;
    w0.h = in / p.s.nomb;
    w0.blk = in - w0.h * p.s.nomb;
    w0.seg = w0.b * hn + in;
  }
  const int total = w0.left;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (elect_one()) {
      prefetch_tmap(&tmKP);
      prefetch_tmap(&tmVP);
      prefetch_tmap(&tmKO);
      prefetch_tmap(&tmVO);
      Walk wk = w0, wv = w0;
      int issued = 0, np = 0, no = 0;
      auto load_tile = [&](Walk& w, const CUtensorMap* mp, const CUtensorMap* mo) -> bool {
        const int key0 = w.key0();
        for (int sp = 0; sp < SPT; ++sp, ++issued) {
          const int s = issued % NSLOT;
          if (issued >= NSLOT && !mbar_wait(slot_empty + s, ((issued / NSLOT) & 1) ^ 1, abort_flag)) return false;
          mbar_arrive_expect_tx(slot_full + s, C::SLOT);
          tma_load_4d(base + s * C::SLOT, w.own ? mo : mp, slot_full + s, 0, key0, sp * CPS,
                      w.own ? w.b * g.Hkv + w.h : w.h);
        }
        w.next();
        return true;
      };
      auto load_k = [&]() -> bool {
        if (wk.first && !wk.own) {
          if (np > 0 && !mbar_wait(qp_empty, (np - 1) & 1, abort_flag)) return false;
          mbar_arrive_expect_tx(qp_full, NCH * p.s.prow * 128);
          for (int c = 0; c < NCH; ++c)
            tma_load_5d(base + C::OFF_QP + c * NP * 128, &tmQP, qp_full, 0, wk.blk % p.s.nmb * NP, c, wk.h,
                        wk.blk / p.s.nmb * p.s.nb);
          ++np;
        } else if (wk.first) {
          const int s = no % QD;
          if (no >= QD && !mbar_wait(qo_empty + s, ((no / QD) & 1) ^ 1, abort_flag)) return false;
          mbar_arrive_expect_tx(qo_full + s, C::QO);
          tma_load_4d(base + C::OFF_QO + s * C::QO, &tmQO, qo_full + s, 0, wk.blk * kOwnRows, 0, wk.b * g.Hkv + wk.h);
          ++no;
        }
        return load_tile(wk, &tmKP, &tmKO);
      };
      // slots in MMA order: K(0), K(1), then per tile n: V(n), K(n + 2)
      bool ok = load_k() && (total < 2 || load_k());
      for (int n = 0; ok && n < total; ++n) ok = load_tile(wv, &tmVP, &tmVO) && (n + 2 >= total || load_k());
      if (*abort_flag) {  // unwinding: the loads in flight land before shared memory is released
        if (np > 0) mbar_wait_drain(qp_full, (np - 1) & 1);
        drain_ring(qo_full, QD, no);
        drain_ring(slot_full, NSLOT, issued);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (elect_one()) {
      const uint32_t idSp = idesc_f16(T, NP, 1, 1, 0, 0), idSo = idesc_f16(T, kOwnRows, 1, 1, 0, 0);  // K x Q^T, both K-major
      const uint32_t idPVp = idesc_f16(T, NP, 1, 1, 1, NP > 16 ? 1 : 0);  // V^T (MN-major) x P^T
      const uint32_t idPVo = idesc_f16(T, kOwnRows, 1, 1, 1, 0);
      Walk ws = w0, wv = w0;
      int used = 0, np = 0, no = 0;
      auto issue_s = [&](int n) -> bool {  // S^T(n) into buffer n & 1
        const int own = ws.own, qs = own ? (no % QD) : 0;
        uint64_t* qf = own ? qo_full + qs : qp_full;
        if (ws.first && !mbar_wait(qf, own ? (no / QD) & 1 : np & 1, abort_flag)) return false;
        const uint64_t qd = smem_desc_sw128(smem_u32(base + (own ? C::OFF_QO + qs * C::QO : C::OFF_QP)), 16, 1024);
        const uint32_t qpitch = (own ? kOwnRows : NP) * 128, idS = own ? idSo : idSp;
        for (int sp = 0; sp < SPT; ++sp, ++used) {
          const int s = used % NSLOT;
          if (!mbar_wait(slot_full + s, (used / NSLOT) & 1, abort_flag)) return false;
          tc_fence_after();
          const uint64_t kd = smem_desc_sw128(smem_u32(base + s * C::SLOT), 16, 1024);
#pragma unroll
          for (int cc = 0; cc < CPS; ++cc) {
            const int c = sp * CPS + cc;
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              mma_ss(tmem + C::S_COL + NP * (n & 1), desc_add(kd, cc * T * 128 + ks * 32),
                     desc_add(qd, c * qpitch + ks * 32), idS, (c | ks) ? 1u : 0u);
          }
          mma_commit(slot_empty + s);
        }
        mma_commit(s_full + (n & 1));
        if (ws.last()) {  // the visit's queries are read
          mma_commit(own ? qo_empty + qs : qp_empty);
          if (own) ++no;
          else ++np;
        }
        ws.next();
        return true;
      };
      bool ok = issue_s(0) && (total < 2 || issue_s(1));
      for (int n = 0; ok && n < total; ++n) {
        if (!mbar_wait(p_full + (n & 1), (n >> 1) & 1, abort_flag)) { ok = false; break; }
        tc_fence_after();
        const int own = wv.own;
        const uint32_t acc = wv.first ? 0u : 1u;
        const uint64_t pd = (NP > 16 && !own) ? smem_desc_sw128(smem_u32(base + C::OFF_P + (n & 1) * C::PB), T * 128, 1024)
                                              : smem_desc_sw128(smem_u32(base + C::OFF_P + (n & 1) * C::PB), 16, 1024);
        // O^T block h (head-dim columns [128 h, 128 h + 128)) += V^T . P^T: one slot a block
        for (int h = 0; h < SPT; ++h, ++used) {
          const int s = used % NSLOT;
          if (!mbar_wait(slot_full + s, (used / NSLOT) & 1, abort_flag)) { ok = false; break; }
          tc_fence_after();
          const uint64_t vd = smem_desc_sw128(smem_u32(base + s * C::SLOT), T * 128, 1024);  // MN-major
          if (NP > 16 && !own) {
#pragma unroll
            for (int ks = 0; ks < T / 16; ++ks)
              mma_ss(tmem + C::O_COL + NP * h, desc_add(vd, ks * 2048), desc_add(pd, ks * 2048), idPVp,
                     (acc || ks > 0) ? 1u : 0u);
          } else {
#pragma unroll
            for (int ks = 0; ks < T / 16; ++ks)
              mma_ss(tmem + C::O_COL + NP * h, desc_add(vd, ks * 2048),
                     desc_add(pd, (ks >> 2) * kOwnRows * 128 + (ks & 3) * 32), idPVo, (acc || ks > 0) ? 1u : 0u);
          }
          mma_commit(slot_empty + s);
        }
        if (!ok) break;
        mma_commit(o_done);
        wv.next();
        if (n + 2 < total && !issue_s(n + 2)) { ok = false; break; }  // after PV(n): S buffer n & 1 is free
      }
      mma_commit(mma_drain);
      mbar_wait_drain(mma_drain, 0);
    }
  } else {
    // ------------------------------------------------------------ softmax
    SoftCtx c;
    c.base = base;
    c.s_full = s_full;
    c.p_full = p_full;
    c.o_done = o_done;
    c.xch = xch;
    c.abort = abort_flag;
    c.tmem = tmem;
    c.n = 0;
    c.xc = 0;
    Walk w = w0;
    bool ok = true;
    while (ok && w.left > 0) ok = w.own ? softmax_visit<D, NP, kOwnRows>(p, w, c) : softmax_visit<D, NP, NP>(p, w, c);
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

// Merge of one query row's partials: those of its prefix block and of its own
// cache, one for each CTA that had a run of the segment.  Rows without a key
// get o = 0 and lse = -inf (or the sink's logit); rows of an empty place of
// the batch are not written.
template <int D>
struct MergeCfg {
  static constexpr int VEC = D >= 128 ? 4 : 2, THREADS = D / VEC;
};
constexpr int kMaxParts = 2 * kSMs;

template <int D>
__global__ void __launch_bounds__(MergeCfg<D>::THREADS) shared_merge_kernel(const SharedParams p) {
  constexpr int VEC = MergeCfg<D>::VEC;
  __shared__ float wts[kMaxParts];
  __shared__ float stat[2];
  const SharedGeom& g = p.g;
  const SharedSplit& s = p.s;
  const int row = blockIdx.x;  // (b Hkv + kv head) M + m
  const int bkv = row / g.M, m = row - bkv * g.M, b = bkv / g.Hkv, h = bkv - b * g.Hkv;
  grid_dependency_wait();
  const int len = p.own_len[b];
  if (len < 0) return;
  const int tp = p.plan[0], units = p.plan[1], ctas = p.plan[2];
  const int nt = own_tiles(g, len), hn = g.Hkv * s.nomb;
  // CTAs c whose run holds a unit u: floor(units c / ctas) <= u
  auto cta_of = [&](int u) { return (int)((((long long)u + 1) * ctas - 1) / units); };
  int np = 0, no = 0;
  const float *pml = nullptr, *po = nullptr, *oml = nullptr, *oo = nullptr;
  if (tp > 0) {
    const int rb = s.nmb > 1 ? b * s.nmb + m / s.np : b / s.nb;
    const int q = s.nmb > 1 ? m % s.np : b % s.nb * g.M + m;
    const int seg = h * s.nrb + rb;
    const int c0 = cta_of(seg * tp);
    np = cta_of(seg * tp + tp - 1) - c0 + 1;
    const size_t at = (size_t)(c0 + seg) * s.prow + q;
    pml = p.pp_ml + at * 2;
    po = p.pp_o + at * D;
  }
  if (nt > 0) {
    const int in = h * s.nomb + m / kOwnRows;
    const int u = g.Hkv * s.nrb * tp + p.plan[kPlanInts + b] * hn + in * nt;
    const int c0 = cta_of(u);
    no = cta_of(u + nt - 1) - c0 + 1;
    const size_t at = (size_t)(c0 + b * hn + in) * s.orow + m % kOwnRows;
    oml = p.po_ml + at * 2;
    oo = p.po_o + at * D;
  }
  const int n = np + no;
  auto ml_of = [&](int i) {
    return *reinterpret_cast<const float2*>(i < np ? pml + (size_t)i * s.prow * 2 : oml + (size_t)(i - np) * s.orow * 2);
  };
  if (threadIdx.x < 32) {
    float mx = -INFINITY;
    for (int i = threadIdx.x; i < n; i += 32) mx = fmaxf(mx, ml_of(i).x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    float l = 0.f;
    for (int i = threadIdx.x; i < n; i += 32) {
      const float2 v = ml_of(i);
      // a part without a visible key adds nothing (its l is 0; NaN scores leave
      // no maximum either, and a NaN l)
      const float w = v.x == -INFINITY ? 0.f : exp2f(v.x - mx);
      wts[i] = w;
      l += v.x == -INFINITY ? v.y : w * v.y;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (threadIdx.x == 0) {
      stat[0] = mx;
      stat[1] = l;
    }
  }
  __syncthreads();
  const float mx = stat[0], l = stat[1];
  const float* sink = p.sinks ? p.sinks + h * g.G + m / g.Lq : nullptr;
  float inv, lse;
  if (mx == -INFINITY && l == 0.f) {
    inv = 0.f;
    lse = sink ? *sink : -INFINITY;
  } else {
    inv = 1.f / l;
    lse = (mx + log2f(l)) * kLn2;
    if (sink) inv = sink_finish(*sink, mx, l, &lse);
  }
  float acc[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
  const int d = threadIdx.x * VEC;
  auto add = [&](const float* src, int cnt, int stride, const float* wt) {
#pragma unroll 4
    for (int i = 0; i < cnt; ++i) {
      const float w = wt[i];
      if constexpr (VEC == 4) {
        const float4 v = *reinterpret_cast<const float4*>(src + (size_t)i * stride * D + d);
        acc[0] = fmaf(w, v.x, acc[0]);
        acc[1] = fmaf(w, v.y, acc[1]);
        acc[2] = fmaf(w, v.z, acc[2]);
        acc[3] = fmaf(w, v.w, acc[3]);
      } else {
        const float2 v = *reinterpret_cast<const float2*>(src + (size_t)i * stride * D + d);
        acc[0] = fmaf(w, v.x, acc[0]);
        acc[1] = fmaf(w, v.y, acc[1]);
      }
    }
  };
  add(po, np, s.prow, wts);
  add(oo, no, s.orow, wts + np);
  uint16_t* dst = p.o + (size_t)row * D + d;
#pragma unroll
  for (int e = 0; e < VEC; e += 2) *reinterpret_cast<uint32_t*>(dst + e) = pack_bf16(acc[e] * inv, acc[e + 1] * inv);
  if (threadIdx.x == 0) p.lse[row] = lse;
}

struct SharedWs {
  size_t plan, pp_ml, pp_o, po_ml, po_o, total;
};
SharedWs shared_ws(const SharedGeom& g) {
  const SharedSplit s = shared_split(g);
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t ps = (size_t)(kSMs + (long long)g.Hkv * s.nrb) * s.prow, os = (size_t)(kSMs + (long long)g.B * g.Hkv * s.nomb) * s.orow;
  SharedWs w;
  w.plan = 0;
  w.pp_ml = w.plan + up(((size_t)g.B + kPlanInts) * 4);
  w.pp_o = w.pp_ml + (g.P > 0 ? up(ps * 8) : 0);
  w.po_ml = w.pp_o + (g.P > 0 ? up(ps * g.D * 4) : 0);
  w.po_o = w.po_ml + up(os * 8);
  w.total = w.po_o + up(os * g.D * 4);
  return w;
}

template <int D, int NP>
cudaError_t shared_d(const SharedGeom& g, const SharedArgs& a, void* ws, int* status, cudaStream_t st) {
  using C = ShCfg<D, NP>;
  const SharedSplit s = shared_split(g);
  CUtensorMap tqp, tqo, tkp, tvp, tko, tvo;
  cudaError_t e;
  if ((e = make_tmap_rows_5d(&tqp, a.q, D, g.M, g.Hkv, g.B, s.mb, s.nb)) != cudaSuccess) return e;
  if ((e = make_tmap_f16_chunks(&tqo, a.q, D, g.M, g.B * g.Hkv, kOwnRows, C::NCH)) != cudaSuccess) return e;
  if ((e = make_tmap_f16_chunks(&tko, a.ko, D, g.own_rows, g.B * g.Hkv, T, C::CPS)) != cudaSuccess) return e;
  if ((e = make_tmap_f16_chunks(&tvo, a.vo, D, g.own_rows, g.B * g.Hkv, T, C::CPS)) != cudaSuccess) return e;
  if (g.P > 0) {
    // rows at or beyond the prefix's length read as zero
    if ((e = make_tmap_f16_chunks(&tkp, a.kp, D, g.P, g.Hkv, T, C::CPS, g.prefix_rows)) != cudaSuccess) return e;
    if ((e = make_tmap_f16_chunks(&tvp, a.vp, D, g.P, g.Hkv, T, C::CPS, g.prefix_rows)) != cudaSuccess) return e;
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
  if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM)) != cudaSuccess)
    return e;
  kern<<<kSMs, kThr, C::SMEM, st>>>(tqp, tqo, tkp, tvp, tko, tvo, p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  // the merge, launched as a programmatic dependent: its blocks are placed
  // while the main grid runs and start when that has completed
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(g.B * g.Hkv * g.M));
  cfg.blockDim = dim3(MergeCfg<D>::THREADS);
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, shared_merge_kernel<D>, p);
}

template <int D>
cudaError_t shared_np(const SharedGeom& g, const SharedArgs& a, void* ws, int* status, cudaStream_t st) {
  return shared_split(g).np == 16 ? shared_d<D, 16>(g, a, ws, status, st) : shared_d<D, 64>(g, a, ws, status, st);
}

}  // namespace

SharedSplit shared_split(const SharedGeom& g) {
  SharedSplit s;
  s.np = (long long)g.B * g.M <= 16 ? 16 : 64;
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
  return units < 1.0e9 && (double)g.B * g.Hkv * g.M < 1.0e9 && (double)g.B * g.Hkv * s.nomb < 1.0e9;
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
