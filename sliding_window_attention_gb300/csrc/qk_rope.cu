// Queries and keys of one projection, normalised per head and rotated by
// position, from the projection's token-major rows to the attention's
// [B, H, L, D] (or into a cache), with the values laid out beside them; and
// the backward, from the attention's fp32 dq, dk, dv to the projection's bf16
// gradient and the gradients of the two learned scales.
//
// Mathematics, for one row x (one token, one head, D elements):
//   n = x r,  r = (mean(x^2) + eps)^(-1/2),   u = n w,   y = R u
// with w the learned scale plus weight_offset and R the rotation of element
// pairs by the angles position * inv_freq[i].  With a_e = w_e cos and b_e the
// partner's scale times +-sin (both fixed for a token), every output element
// is y_e = r (x_e a_e + x_partner(e) b_e): one pass over the row in registers.
// Backward, with g = R^T dy and h = g w:
//   dw = sum over rows of g n,   dx = r (h - n mean(h n)).
//
// Angles.  position * frequency loses its fraction in fp32 for far positions
// (half an ulp at 1e6 radians is 0.03), so frequencies come as doubles and a
// CTA turns each once into a 64-bit fixed-point fraction of a full turn;
// position times that fraction, modulo 2^64, loses nothing more (integer
// multiplication wraps as angles do).  The step carries the rounding of two
// fp64 factors and their product, 2^-52 of the turns made at most, and
// sincospif takes the phase's top 32 bits as a float: 2^-26 of a turn.
//
// All sums, the norm and the rotation are fp32; the only rounding to fewer
// bits is the one of each output to bf16 (half a step, 2^-8 of the value).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "swa_internal.h"
#include "tc_ptx.cuh"

namespace swa {
namespace {

constexpr int kThr = 256;

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t bf_pack(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// Frequency (radians a position) as a fraction of a turn, mod 1, in units of 2^-64.
__device__ __forceinline__ uint64_t turn_step(double f) {
  double t = f * 0.15915494309189533577;  // 1 / (2 pi)
  t -= floor(t);
  return __double2ull_rz(t * 18446744073709551616.0);
}
// cos and sin of position * frequency.
__device__ __forceinline__ float2 turn_cs(long long pos, uint64_t step) {
  const uint64_t phase = (uint64_t)pos * step;
  const float half_turns = (float)(int32_t)(uint32_t)(phase >> 32) * 4.656612873077392578125e-10f;  // 2^-31
  float s, c;
  sincospif(half_turns, &s, &c);
  return make_float2(c, s);
}

// Where a token's rotation angles come from.
struct RopePos {
  const double* inv_freq;  // [pairs]
  const int* positions;    // [B, L] or null
  const int* kv_len;       // [B] or null: the tokens are the last L of kv_len[b]
  int pos0, pairs, interleaved;
};
__device__ __forceinline__ long long token_pos(const RopePos& a, int b, int l, int L) {
  if (a.positions) return a.positions[(size_t)b * L + l];
  return (long long)a.pos0 + l + (a.kv_len ? (long long)a.kv_len[b] - L : 0);
}

// Rows staged through shared memory by TMA.  Both directions do a few
// multiplications a byte, so what bounds them is the memory's latency: the
// bytes in flight.  A CTA keeps a ring of stages filled -- a stage is 512 / D
// heads of 8 consecutive tokens, x as the projection laid it out
// ([token][head][D]) and, in the backward, dy as the attention did
// ([head][token][D]); the boxes of two tensor maps -- and its eight warps, one
// a token, work from there.  The stages' units (token group, block of heads)
// form one list that the CTAs share out evenly.  The forward's groups run over
// the whole batch's tokens, so that a generation step of 64 requests is 8
// groups; the backward's stay within a batch entry (dy's layout).
//
// A lane holds E = 8 (16 at D = 512) elements of a row in NG groups of 4, D / NG
// apart: with the whole head rotated in halves an element's partner is then in
// the same lane, and a warp's loads of a group are contiguous.
//
// With few heads a stage of 512 / D heads is mostly empty, so there is a second
// form with a quarter of the heads and four tokens a warp (TPW), which serves
// the shapes whose stages it makes fewer (65,536 tokens, 2 + 1 + 1 heads, D = 64:
// forward 29.7 us, with one token a warp 54.6; backward 34.6 and 71.4).
constexpr int kTok = 8;  // consumer warps, each with TPW tokens of a stage

template <int D, int TPW>
struct StCfg {
  static constexpr int HB = 512 / D / TPW;  // heads of a stage
  static constexpr int E = D == 512 ? 16 : 8;
  static constexpr int NG = E / 4, GS = D / NG;
  static constexpr int LPR = D / E, RPW = 32 / LPR, ITER = HB * TPW / RPW;  // a warp's rows: RPW at a time
  static constexpr int TOKS = kTok * TPW;
  static constexpr int XB = kTok * 512 * 2, YB = kTok * 512 * 4;
};

// The order of a CTA's stages: units [u0, u1) of groups x (Hq, Hkv, Hkv heads in blocks).
struct StList {
  int nq, nk, nv, per;     // blocks of q, k, v heads, and of a group
  int groups, gl;          // token groups, and (backward) those of a batch entry
  __device__ __forceinline__ void split(int cta, int ctas, int& u0, int& u1) const {
    const long long u = (long long)groups * per;
    u0 = (int)(u * cta / ctas);
    u1 = (int)(u * (cta + 1) / ctas);
  }
};

struct StRope {
  StList list;
  RopePos pos;
  const float *wq, *wk;
  uint16_t *qo, *ko, *vo;         // forward outputs
  uint16_t *gq, *gk, *gv;         // backward outputs, token-major
  long long gq_tok, gk_tok, gv_tok;
  float* part;                    // [gridDim.x][2][D] partial dw
  int B, L, Hq, Hkv, kv_rows;
  float eps, off;
  int pass;                       // inputs are the first to leave L2
  int* status;
};

// How a pair is laid out: neighbours; the halves of the whole head (both in
// one lane); the halves of its first 2 * pairs elements (the partner's row
// group is read from shared memory).
enum : int { kInter = 0, kHalves = 1, kPart = 2 };

// Elements are held as pairs of neighbours (.f32x2 arithmetic: one
// instruction for two elements).
__device__ __forceinline__ void ld_bf4(const uint16_t* p, uint64_t* x) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  x[0] = tc::f2_pack(bf_lo(v.x), bf_hi(v.x));
  x[1] = tc::f2_pack(bf_lo(v.y), bf_hi(v.y));
}
__device__ __forceinline__ void ld_f4(const float* p, uint64_t* x) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  x[0] = tc::f2_pack(v.x, v.y);
  x[1] = tc::f2_pack(v.z, v.w);
}
__device__ __forceinline__ uint32_t bf_pack2(uint64_t x) {
  const float2 v = tc::f2_unpack(x);
  return bf_pack(v.x, v.y);
}
__device__ __forceinline__ uint64_t f2_dup(float x) { return tc::f2_pack(x, x); }
__device__ __forceinline__ float f2_sum(uint64_t x) {
  const float2 v = tc::f2_unpack(x);
  return v.x + v.y;
}

// The partners' elements of a row whose own elements are in registers; ld(d,
// v) loads elements d .. d + 3 of the row.
template <int D, int MODE, typename F>
__device__ __forceinline__ void row_partners(const uint64_t (&own)[StCfg<D, 1>::E / 2], uint64_t (&other)[StCfg<D, 1>::E / 2],
                                             int d4, int pairs, F&& ld) {
  using C = StCfg<D, 1>;
  constexpr int W = C::E / 2;
  if constexpr (MODE == kInter) {
#pragma unroll
    for (int e = 0; e < W; ++e) {
      const float2 v = tc::f2_unpack(own[e]);
      other[e] = tc::f2_pack(v.y, v.x);
    }
  } else if constexpr (MODE == kHalves) {
#pragma unroll
    for (int e = 0; e < W; ++e) other[e] = own[(e + W / 2) % W];
  } else {
#pragma unroll
    for (int g = 0; g < C::NG; ++g) {
      const int d = C::GS * g + d4;
      ld(d < pairs ? d + pairs : (d < 2 * pairs ? d - pairs : d), other + 2 * g);
    }
  }
}
// cos, and +-sin as y_e = cos u_e + s_e u_partner(e), of the lane's elements.
template <int D, int MODE>
__device__ __forceinline__ void lane_angles(const float2* cs, int d4, int pairs, uint64_t (&c)[StCfg<D, 1>::E / 2],
                                            uint64_t (&s)[StCfg<D, 1>::E / 2]) {
  using C = StCfg<D, 1>;
  // pairs i, i + 1 as {cos, sin, cos, sin}; beyond the rotated part {1, 0}
  auto two = [&](int i, bool in) {
    return in ? *reinterpret_cast<const float4*>(cs + i) : make_float4(1.f, 0.f, 1.f, 0.f);
  };
  if constexpr (MODE == kHalves) {
    constexpr int H = C::E / 4;  // words of the lower half
#pragma unroll
    for (int g = 0; g < C::NG / 2; ++g)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 v = two(C::GS * g + d4 + 2 * i, true);
        c[2 * g + i] = c[H + 2 * g + i] = tc::f2_pack(v.x, v.z);
        s[2 * g + i] = tc::f2_pack(-v.y, -v.w);
        s[H + 2 * g + i] = tc::f2_pack(v.y, v.w);
      }
  } else {
#pragma unroll
    for (int g = 0; g < C::NG; ++g) {
      const int d = C::GS * g + d4;
      const bool in = d < 2 * pairs, lo = d < pairs;
      if constexpr (MODE == kInter) {
        const float4 v = two(d / 2, in);
        c[2 * g] = tc::f2_pack(v.x, v.x);
        s[2 * g] = tc::f2_pack(-v.y, v.y);
        c[2 * g + 1] = tc::f2_pack(v.z, v.z);
        s[2 * g + 1] = tc::f2_pack(-v.w, v.w);
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float4 v = two((lo ? d : d - pairs) + 2 * i, in);
          c[2 * g + i] = tc::f2_pack(v.x, v.z);
          s[2 * g + i] = lo ? tc::f2_pack(-v.y, -v.w) : tc::f2_pack(v.y, v.w);
        }
      }
    }
  }
}

// Shared memory of a staged kernel: NS stages, then weights, turn steps, the
// warps' cos / sin tables and the barriers.
template <int D, bool BWD, int TPW>
struct StSmem {
  using C = StCfg<D, TPW>;
  static constexpr int STAGE = C::XB + (BWD ? C::YB : 0);
  // stages and CTAs an SM: 96 KB (forward) and 192 KB (backward) in flight;
  // measured at 30,553 tokens, D = 256, 2 x 8 stages of 8 KB take 349 us, 2 x 4
  // 327, 3 x 4 324, 4 x 4 351 (and 3 x 4 is best at 8,192 tokens, D = 128: 13.1
  // us against 14.3 and 15.8); the backward at 16,384 tokens, D = 512, takes 382
  // us with 8 stages of 24 KB, 389 with 5, 518 with 3
  static constexpr int NS = BWD ? (D == 512 ? 8 : (TPW > 1 && D == 128 ? 3 : 4)) : (TPW > 1 ? 6 : 4);
  static constexpr int OFF_W = NS * STAGE;              // [2][D] scales
  static constexpr int OFF_STEP = OFF_W + 2 * D * 4;    // [D / 2]
  static constexpr int OFF_CS = OFF_STEP + D / 2 * 8;   // [tokens][D / 2]
  static constexpr int OFF_BAR = OFF_CS + C::TOKS * D / 2 * 8;
  static constexpr size_t BYTES = (size_t)OFF_BAR + 256 + 128;
  static constexpr int CTAS = BWD ? (D == 512 ? 1 : 2) : (D == 512 || TPW > 1 ? 2 : 3);  // per SM (there 3 would spill)
  static_assert(CTAS * BYTES <= 228 * 1024 - CTAS * 1024, "shared memory");
  static_assert(D / 2 <= kThr, "a frequency a thread");
  static_assert(NS <= kTok, "each warp loads one of the first stages");
  static_assert(!BWD || NS * STAGE >= kTok * D * 4, "the scales' gradients are reduced in the stages");
};

template <int D, int MODE, bool BWD, int TPW>
__global__ void __launch_bounds__(kThr, StSmem<D, BWD, TPW>::CTAS)
    qk_rope_staged_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                          const __grid_constant__ CUtensorMap tmV,   // forward: v's rows
                          const __grid_constant__ CUtensorMap tmDQ, const __grid_constant__ CUtensorMap tmDK,
                          const __grid_constant__ CUtensorMap tmDV, const __grid_constant__ StRope p) {
  using C = StCfg<D, TPW>;
  using M = StSmem<D, BWD, TPW>;
  constexpr int E = C::E, W = E / 2, NG = C::NG, GS = C::GS, HB = C::HB, NS = M::NS, IT = C::ITER;
  constexpr int AI = TPW > 1 ? IT : 1;  // tokens of a lane
  extern __shared__ unsigned char smem_raw[];
  unsigned char* base = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
  float* sw = reinterpret_cast<float*>(base + M::OFF_W);
  uint64_t* step = reinterpret_cast<uint64_t*>(base + M::OFF_STEP);
  uint64_t* full = reinterpret_cast<uint64_t*>(base + M::OFF_BAR);  // [NS]
  uint64_t* empty = full + NS;                                      // [NS]
  volatile int* abort_flag = reinterpret_cast<volatile int*>(empty + NS);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, pairs = p.pos.pairs;
  const StList& ls = p.list;
  tc::grid_launch_dependents();  // dependents wait for this grid's end
  int u0, u1;
  ls.split(blockIdx.x, gridDim.x, u0, u1);

  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      tc::mbar_init(full + i, 1);
      tc::mbar_init(empty + i, kTok);
    }
    *abort_flag = 0;
    tc::fence_mbar_init();
  }
  __syncthreads();
  tc::grid_dependency_wait();

  uint64_t accq[BWD ? W : 1], acck[BWD ? W : 1];  // dw of the lane's elements
#pragma unroll
  for (int e = 0; e < (BWD ? W : 1); ++e) accq[e] = acck[e] = f2_dup(0.f);

  // Stage n (unit u0 + n) is loaded by lane 0 of warp n % kTok, once every
  // warp has consumed stage n - NS; a warp gets to that after its own stage
  // n - NS + 1, so it seldom waits.
  int loaded = -1;  // the last stage this thread loaded
  const uint64_t policy = tc::l2_policy(p.pass);
  auto load = [&](int n) {
    const int s = n % NS, u = u0 + n, grp = u / ls.per, i = u - grp * ls.per;
    if (n >= NS && !tc::mbar_wait(empty + s, ((n / NS) & 1) ^ 1, abort_flag)) return;
    const int b = BWD ? grp / ls.gl : 0, l0 = (grp - b * ls.gl) * C::TOKS;  // forward: tokens of the whole batch
    const int kind = i < ls.nq ? 0 : (i < ls.nq + ls.nk ? 1 : 2);
    const int h0 = (i - (kind > 0 ? ls.nq : 0) - (kind > 1 ? ls.nk : 0)) * HB;
    unsigned char* x = base + s * M::STAGE;
    // D = 512 rows are two halves of 256 (a box is at most 256 wide)
    const bool has_x = !BWD || kind < 2;
    tc::mbar_arrive_expect_tx(full + s, (has_x ? C::XB : 0) + (BWD ? C::YB : 0));
    if (has_x) tc::tma_load_4d(x, kind == 0 ? &tmQ : (kind == 1 ? &tmK : &tmV), full + s, 0, D == 512 ? 2 * h0 : h0, l0, b, policy);
    if (BWD) {
      const CUtensorMap* m = kind == 0 ? &tmDQ : (kind == 1 ? &tmDK : &tmDV);
      if (D == 512) tc::tma_load_5d(x + C::XB, m, full + s, 0, 0, l0, h0, b, policy);
      else tc::tma_load_4d(x + C::XB, m, full + s, 0, l0, h0, b, policy);
    }
    loaded = n;
  };
  // Frequencies and scales are asked for before the stages: behind the first
  // stages of every CTA (29 MB) they would take 4 us.
  constexpr int WN = (2 * D + kThr - 1) / kThr;
  const double freq = threadIdx.x < pairs ? p.pos.inv_freq[threadIdx.x] : 0.0;
  float wr[WN];
#pragma unroll
  for (int j = 0; j < WN; ++j) {
    const int i = threadIdx.x + j * kThr;
    const float* w = i < D ? p.wq : p.wk;
    wr[j] = i < 2 * D && w ? w[i < D ? i : i - D] + p.off : 1.f;
  }
  asm volatile("" ::: "memory");
  if (lane == 0 && warp < NS && warp < u1 - u0) load(warp);
  if (threadIdx.x < pairs) step[threadIdx.x] = turn_step(freq);
#pragma unroll
  for (int j = 0; j < WN; ++j)
    if (threadIdx.x + j * kThr < 2 * D) sw[threadIdx.x + j * kThr] = wr[j];
  __syncthreads();

  {
    float2* cs = reinterpret_cast<float2*>(base + M::OFF_CS) + warp * TPW * (D / 2);
    const int sub = lane / C::LPR, d4 = 4 * (lane % C::LPR);
    int u = u0, slot = 0, grp = u0 / ls.per, skip = u0 - grp * ls.per;  // blocks of the group before this CTA's
    uint32_t phase = 0;
    bool ok = true;
    // The stages of one kind's nb head blocks: f(stage, first head) works on one.
    auto blocks = [&](int nb, auto&& f) {
      int blk = min(skip, nb);
      skip -= blk;
      for (; blk < nb && u < u1; ++blk, ++u) {
        if (!__all_sync(0xffffffffu, tc::mbar_wait(full + slot, phase, abort_flag))) {
          ok = false;
          return;
        }
        f(base + slot * M::STAGE, blk * HB);
        __syncwarp();
        if (lane == 0) {
          tc::mbar_arrive(empty + slot);
          const int n = u - u0 + NS - 1;
          if (n % kTok == warp && n >= NS && n < u1 - u0) load(n);
        }
        __syncwarp();
        if (++slot == NS) {
          slot = 0;
          phase ^= 1;
        }
      }
    };
    for (; ok && u < u1; ++grp) {
      // token i of this warp: its batch entry and place there
      auto token = [&](int i, int& b, int& l) {
        const int t = grp * C::TOKS + warp * TPW + i;
        b = BWD ? grp / ls.gl : t / p.L;
        l = BWD ? t - b * ls.gl * C::TOKS : t - b * p.L;
        return b < p.B && l < p.L;
      };
      __syncwarp();
#pragma unroll 1
      for (int i = 0; i < TPW; ++i) {
        int b, l;
        if (!token(i, b, l)) break;
        const long long pos = token_pos(p.pos, b, l, p.L);
        for (int k = lane; k < pairs; k += 32) cs[i * (D / 2) + k] = turn_cs(pos, step[k]);
      }
      __syncwarp();
      // this lane's tokens: of its row in each round (TPW > 1), or the warp's
      bool live[AI];
      int tb[AI], tl[AI];
#pragma unroll
      for (int i = 0; i < AI; ++i) live[i] = token(TPW > 1 ? (i * C::RPW + sub) / HB : 0, tb[i], tl[i]);
      auto table = [&](int i) { return cs + (TPW > 1 ? (i * C::RPW + sub) / HB * (D / 2) : 0); };
      auto head = [&](int it) { return TPW > 1 ? (it * C::RPW + sub) % HB : it * C::RPW + sub; };
      uint64_t a[AI][W], q[AI][W];  // cos and +-sin (forward: times the element's and its partner's scale)
      if constexpr (!BWD) {
        // q or k rows: at = the tokens' rows of head 0, heads `pitch` elements apart
        auto rows = [&](int nb, int H, const float* w, uint16_t* out, const long long (&at)[AI], long long pitch,
                        const bool (&store)[AI]) {
          {
            uint64_t wv[W], wp[W];
#pragma unroll
            for (int g = 0; g < NG; ++g) ld_f4(w + GS * g + d4, wv + 2 * g);
            row_partners<D, MODE>(wv, wp, d4, pairs, [&](int d, uint64_t* v) { ld_f4(w + d, v); });
#pragma unroll
            for (int i = 0; i < AI; ++i) {
              lane_angles<D, MODE>(table(i), d4, pairs, a[i], q[i]);
#pragma unroll
              for (int e = 0; e < W; ++e) {
                a[i][e] = tc::f2_mul(a[i][e], wv[e]);
                q[i][e] = tc::f2_mul(q[i][e], wp[e]);
              }
            }
          }
          blocks(nb, [&](const unsigned char* st, int h0) {
            const uint16_t* xs = reinterpret_cast<const uint16_t*>(st) + warp * 512 + sub * D;  // [token][head][D]
            uint64_t f[IT][W], o[IT][W];
            float ss[IT];
#pragma unroll
            for (int it = 0; it < IT; ++it) {
              const uint16_t* x = xs + it * C::RPW * D;
#pragma unroll
              for (int g = 0; g < NG; ++g) ld_bf4(x + GS * g + d4, f[it] + 2 * g);
              row_partners<D, MODE>(f[it], o[it], d4, pairs, [&](int d, uint64_t* v) { ld_bf4(x + d, v); });
              uint64_t t = tc::f2_mul(f[it][0], f[it][0]);
#pragma unroll
              for (int e = 1; e < W; ++e) t = tc::f2_fma(f[it][e], f[it][e], t);
              ss[it] = f2_sum(t);
            }
#pragma unroll
            for (int k = C::LPR / 2; k > 0; k >>= 1)
#pragma unroll
              for (int it = 0; it < IT; ++it) ss[it] += __shfl_xor_sync(0xffffffffu, ss[it], k);
#pragma unroll
            for (int it = 0; it < IT; ++it) {
              const int h = h0 + head(it), i = TPW > 1 ? it : 0;
              const uint64_t rn = f2_dup(rsqrtf(ss[it] * (1.f / D) + p.eps));
#pragma unroll
              for (int e = 0; e < W; ++e)
                f[it][e] = tc::f2_mul(rn, tc::f2_fma(f[it][e], a[i][e], tc::f2_mul(o[it][e], q[i][e])));
              if (store[i] && h < H) {
                uint16_t* dst = out + at[i] + h * pitch + d4;
#pragma unroll
                for (int g = 0; g < NG; ++g)
                  *reinterpret_cast<uint2*>(dst + GS * g) = make_uint2(bf_pack2(f[it][2 * g]), bf_pack2(f[it][2 * g + 1]));
              }
            }
          });
        };
        bool kv_ok[AI];
        long long q_at[AI], kv_at[AI];
#pragma unroll
        for (int i = 0; i < AI; ++i) {
          const int b = tb[i], l = tl[i], row = p.pos.kv_len ? (live[i] ? p.pos.kv_len[b] - p.L + l : -1) : l;
          kv_ok[i] = live[i] && row >= 0 && row < p.kv_rows;  // rows outside the cache are not written
          q_at[i] = ((long long)b * p.Hq * p.L + l) * D;
          kv_at[i] = ((long long)b * p.Hkv * p.kv_rows + row) * D;
        }
        const long long kv_pitch = (long long)p.kv_rows * D;
        rows(ls.nq, p.Hq, sw, p.qo, q_at, (long long)p.L * D, live);
        if (ok && ls.nk) rows(ls.nk, p.Hkv, sw + D, p.ko, kv_at, kv_pitch, kv_ok);
        if (ok && ls.nv)
          blocks(ls.nv, [&](const unsigned char* st, int h0) {
            const uint16_t* xs = reinterpret_cast<const uint16_t*>(st) + warp * 512 + sub * D;
#pragma unroll
            for (int it = 0; it < IT; ++it) {
              const int h = h0 + head(it), i = TPW > 1 ? it : 0;
              if (!kv_ok[i] || h >= p.Hkv) continue;
#pragma unroll
              for (int g = 0; g < NG; ++g)
                *reinterpret_cast<uint2*>(p.vo + kv_at[i] + h * kv_pitch + GS * g + d4) =
                    *reinterpret_cast<const uint2*>(xs + it * C::RPW * D + GS * g + d4);
            }
          });
      } else {
        // rows of dy: [head][token][D]
        auto dy_at = [&](const unsigned char* st, int it) {
          const int tok = warp * TPW + (TPW > 1 ? (it * C::RPW + sub) / HB : 0);
          return reinterpret_cast<const float*>(st + C::XB) + (head(it) * C::TOKS + tok) * D;
        };
        long long tok[AI];
#pragma unroll
        for (int i = 0; i < AI; ++i) {
          tok[i] = (long long)tb[i] * p.L + tl[i];
          lane_angles<D, MODE>(table(i), d4, pairs, a[i], q[i]);
#pragma unroll
          for (int e = 0; e < W; ++e) q[i][e] = tc::f2_mul(q[i][e], f2_dup(-1.f));  // the rotation's transpose
        }
        auto rows = [&](int nb, int H, const float* w, uint16_t* out, long long pitch, uint64_t (&acc)[W]) {
          uint64_t we[W];
#pragma unroll
          for (int g = 0; g < NG; ++g) ld_f4(w + GS * g + d4, we + 2 * g);
          blocks(nb, [&](const unsigned char* st, int h0) {
            const uint16_t* xs = reinterpret_cast<const uint16_t*>(st) + warp * 512 + sub * D;  // [token][head][D]
            uint64_t f[IT][W], y[IT][W];
            float ss[IT], dot[IT];
#pragma unroll
            for (int it = 0; it < IT; ++it) {
              const uint16_t* x = xs + it * C::RPW * D;
              const float* dy = dy_at(st, it);
              const int i = TPW > 1 ? it : 0;
              uint64_t o[W];
#pragma unroll
              for (int g = 0; g < NG; ++g) {
                ld_f4(dy + GS * g + d4, y[it] + 2 * g);
                ld_bf4(x + GS * g + d4, f[it] + 2 * g);
              }
              row_partners<D, MODE>(y[it], o, d4, pairs, [&](int d, uint64_t* v) { ld_f4(dy + d, v); });
              uint64_t t = f2_dup(0.f), v = f2_dup(0.f);
#pragma unroll
              for (int e = 0; e < W; ++e) {
                y[it][e] = tc::f2_fma(a[i][e], y[it][e], tc::f2_mul(q[i][e], o[e]));
                t = tc::f2_fma(f[it][e], f[it][e], t);
                v = tc::f2_fma(tc::f2_mul(y[it][e], we[e]), f[it][e], v);
              }
              ss[it] = f2_sum(t);
              dot[it] = f2_sum(v);
            }
#pragma unroll
            for (int k = C::LPR / 2; k > 0; k >>= 1)
#pragma unroll
              for (int it = 0; it < IT; ++it) {
                ss[it] += __shfl_xor_sync(0xffffffffu, ss[it], k);
                dot[it] += __shfl_xor_sync(0xffffffffu, dot[it], k);
              }
#pragma unroll
            for (int it = 0; it < IT; ++it) {
              const int h = h0 + head(it), i = TPW > 1 ? it : 0;
              if (!live[i] || h >= H) continue;
              const float r = rsqrtf(ss[it] * (1.f / D) + p.eps);
              const uint64_t rn = f2_dup(r), m = f2_dup(-dot[it] * r * r * (1.f / D));  // -mean(h n) r
              uint16_t* dst = out + tok[i] * pitch + (long long)h * D + d4;
#pragma unroll
              for (int e = 0; e < W; ++e) {
                acc[e] = tc::f2_fma(tc::f2_mul(y[it][e], rn), f[it][e], acc[e]);
                y[it][e] = tc::f2_mul(rn, tc::f2_fma(f[it][e], m, tc::f2_mul(y[it][e], we[e])));
              }
#pragma unroll
              for (int g = 0; g < NG; ++g)
                *reinterpret_cast<uint2*>(dst + GS * g) = make_uint2(bf_pack2(y[it][2 * g]), bf_pack2(y[it][2 * g + 1]));
            }
          });
        };
        rows(ls.nq, p.Hq, sw, p.gq, p.gq_tok, accq);
        if (ok && ls.nk) rows(ls.nk, p.Hkv, sw + D, p.gk, p.gk_tok, acck);
        if (ok && ls.nv)
          blocks(ls.nv, [&](const unsigned char* st, int h0) {
#pragma unroll
            for (int it = 0; it < IT; ++it) {
              const int h = h0 + head(it), i = TPW > 1 ? it : 0;
              if (!live[i] || h >= p.Hkv) continue;
              uint16_t* dst = p.gv + tok[i] * p.gv_tok + (long long)h * D + d4;
#pragma unroll
              for (int g = 0; g < NG; ++g) {
                uint64_t v[2];
                ld_f4(dy_at(st, it) + GS * g + d4, v);
                *reinterpret_cast<uint2*>(dst + GS * g) = make_uint2(bf_pack2(v[0]), bf_pack2(v[1]));
              }
            }
          });
      }
    }
  }

  if (*abort_flag && loaded >= 0) tc::mbar_wait_drain(full + loaded % NS, (loaded / NS) & 1);  // a load may be in flight
  __syncthreads();
  if (*abort_flag) {
    if (threadIdx.x == 0) atomicCAS(p.status, 0, kStatusTimeout);
    return;
  }
  if constexpr (BWD) {
    // this CTA's dw: a warp's row slots, then the warps, in a fixed order (in
    // the stages' memory: every load has been consumed)
    float* red = reinterpret_cast<float*>(base);  // [kTok][D]
    const int sub = lane / C::LPR, d4 = 4 * (lane % C::LPR);
#pragma unroll
    for (int kind = 0; kind < 2; ++kind) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float2 pr = tc::f2_unpack(kind ? acck[e / 2] : accq[e / 2]);
        float v = e & 1 ? pr.y : pr.x;
#pragma unroll
        for (int o = C::LPR; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (sub == 0) red[warp * D + GS * (e >> 2) + d4 + (e & 3)] = v;
      }
      __syncthreads();
      for (int d = threadIdx.x; d < D; d += kThr) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kTok; ++w) v += red[w * D + d];
        p.part[((size_t)blockIdx.x * 2 + kind) * D + d] = v;
      }
      __syncthreads();
    }
  }
}

// dw[kind][d] = sum of the CTAs' partials (at most 2 a SM): 32 strided sums a column, then those.
constexpr int kDwLoads = (2 * 152 + 31) / 32;
__global__ void __launch_bounds__(1024) qk_rope_dw_kernel(const float* part, float* dwq, float* dwk, int D, int n) {
  __shared__ float red[32][33];
  const int x = threadIdx.x & 31, grp = threadIdx.x >> 5, col = blockIdx.x * 32 + x;  // column of [2][D]
  tc::grid_launch_dependents();
  tc::grid_dependency_wait();
  float t[kDwLoads], v = 0.f;  // every load of a thread is under way at once
#pragma unroll
  for (int i = 0; i < kDwLoads; ++i) {
    const int c = grp + 32 * i;
    t[i] = c < n ? part[(size_t)c * 2 * D + col] : 0.f;
  }
#pragma unroll
  for (int i = 0; i < kDwLoads; ++i) v += t[i];
  red[grp][x] = v;
  __syncthreads();
  v = red[x][grp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (x == 0) {
    const int c = blockIdx.x * 32 + grp;
    float* out = c < D ? dwq : dwk;
    if (out) out[c < D ? c : c - D] = v;
  }
}

RopePos rope_pos(const RopeArgs& a) {
  RopePos r;
  r.inv_freq = a.inv_freq;
  r.positions = a.positions;
  r.kv_len = a.kv_len;
  r.pos0 = a.pos0;
  r.pairs = a.rot_dim / 2;
  r.interleaved = a.interleaved;
  return r;
}

// The stages' units with TPW tokens a warp.
StList stage_list(const RopeArgs& a, bool v, bool bwd, int tpw) {
  StList l;
  const int hb = 512 / a.D / tpw, toks = kTok * tpw;
  l.nq = (a.Hq + hb - 1) / hb;
  l.nk = a.k ? (a.Hkv + hb - 1) / hb : 0;
  l.nv = v ? (a.Hkv + hb - 1) / hb : 0;
  l.per = l.nq + l.nk + l.nv;
  l.gl = bwd ? (a.L + toks - 1) / toks : 0;
  l.groups = bwd ? a.B * l.gl : (int)(((long long)a.B * a.L + toks - 1) / toks);
  return l;
}
// Four tokens a warp where that halves the stages and leaves one for every CTA
// (forward: two; 8,192 tokens, 2 + 1 + 1 heads, D = 64: 8.3 us, else 10.1; but at
// 4,096 tokens 7.5, else 7.1), or makes a quarter fewer of very many (30,000
// tokens, 8 + 4 + 4 heads, D = 64: 24.2 us, else 28.1; but at 4,096 8.6, else 7.2).
int tokens_a_warp(const RopeArgs& a, bool v, bool bwd) {
  if (a.D > 128) return 1;
  const StList one = stage_list(a, v, bwd, 1), four = stage_list(a, v, bwd, 4);
  const long long u1 = (long long)one.groups * one.per, u4 = (long long)four.groups * four.per;
  const bool fewer = 2 * u4 <= u1 ? u4 >= (bwd ? 2 : 4) * 152 : 4 * u4 <= 3 * u1 && u4 >= 16 * 152;
  return fewer && four.groups < (1 << 26) ? 4 : 1;  // (32-bit token indexes)
}

StRope staged_params(const RopeArgs& a, bool v, bool bwd, int* status) {
  StRope p = {};
  p.pos = rope_pos(a);
  p.wq = a.wq;
  p.wk = a.wk;
  p.B = a.B;
  p.L = a.L;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.eps = a.eps;
  p.off = a.weight_offset;
  p.status = status;
  // Where the outputs take at most half of L2, and inputs and outputs more than
  // it can hold beside other data, the inputs give way: the outputs then stay for
  // the kernel that reads them next and are not written out meanwhile.  Backward,
  // 32 + 4 + 4 heads, D = 512, with and without, at 1,024 tokens (42 MB of outputs):
  // 28.7 and 32.3 us; forward, 32 + 16 + 16 heads, D = 256, at 2,048 (67 MB): 20.8
  // and 22.6; backward, 8 + 4 + 4 heads, D = 128, at 24,576 (100 MB): 64.7 and 62.0; at
  // 2,048 (8 MB): 10.0 and 9.3.
  const double out = (double)a.B * a.L * (a.Hq + (a.k ? a.Hkv : 0) + (v ? a.Hkv : 0)) * a.D * 2, in = bwd ? 2.75 * out : out;
  p.pass = out <= 68.0e6 && in + out > 48.0e6;
  return p;
}

template <int D, bool BWD, int TPW>
int staged_ctas(const StList& l) {
  const long long u = (long long)l.groups * l.per, most = 152 * StSmem<D, BWD, TPW>::CTAS;
  return (int)(u < most ? u : most);
}
template <int D, int MODE, bool BWD, int TPW>
cudaError_t staged_mode(const StRope& p, const CUtensorMap (&m)[6], int grid, cudaStream_t s) {
  auto kern = qk_rope_staged_kernel<D, MODE, BWD, TPW>;
  const size_t smem = StSmem<D, BWD, TPW>::BYTES;
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = allow_smem(kern, (int)smem, done);
  if (e != cudaSuccess) return e;
  return launch_dependent(kern, dim3(grid), dim3(kThr), smem, s, m[0], m[1], m[2], m[3], m[4], m[5], p);
}

template <int D, bool BWD, int TPW>
cudaError_t staged_launch(const StRope& p, const CUtensorMap (&m)[6], int grid, cudaStream_t s) {
  if (p.pos.interleaved) return staged_mode<D, kInter, BWD, TPW>(p, m, grid, s);
  return 2 * p.pos.pairs == D ? staged_mode<D, kHalves, BWD, TPW>(p, m, grid, s)
                              : staged_mode<D, kPart, BWD, TPW>(p, m, grid, s);
}

template <int D, int TPW>
cudaError_t staged_fwd(const RopeArgs& a, const uint16_t* v, long long v_tok, StRope& p, cudaStream_t s) {
  using C = StCfg<D, TPW>;
  p.list = stage_list(a, v != nullptr, false, TPW);
  CUtensorMap m[6];
  const int toks = a.B * a.L;
  cudaError_t e = make_tmap_tokens(&m[0], a.q, D, a.Hq, toks, 1, a.q_tok, C::TOKS, C::HB);
  if (e == cudaSuccess && a.k) e = make_tmap_tokens(&m[1], a.k, D, a.Hkv, toks, 1, a.k_tok, C::TOKS, C::HB);
  if (e == cudaSuccess && v) e = make_tmap_tokens(&m[2], v, D, a.Hkv, toks, 1, v_tok, C::TOKS, C::HB);
  if (e != cudaSuccess) return e;
  if (!a.k) m[1] = m[0];  // not read
  if (!v) m[2] = m[0];
  m[3] = m[4] = m[5] = m[0];
  const int grid = staged_ctas<D, false, TPW>(p.list);
  return staged_launch<D, false, TPW>(p, m, grid, s);
}

template <int D, int TPW>
cudaError_t staged_bwd(const RopeArgs& a, const float* dq, const float* dk, const float* dv, StRope& p, float* dwq,
                       float* dwk, cudaStream_t s) {
  using C = StCfg<D, TPW>;
  p.list = stage_list(a, dv != nullptr, true, TPW);
  CUtensorMap m[6];
  cudaError_t e = make_tmap_tokens(&m[0], a.q, D, a.Hq, a.L, a.B, a.q_tok, C::TOKS, C::HB);
  if (e == cudaSuccess) e = make_tmap_f32_tokens(&m[3], dq, D, a.Hq, a.L, a.B, C::TOKS, C::HB);
  if (e == cudaSuccess && a.k) e = make_tmap_tokens(&m[1], a.k, D, a.Hkv, a.L, a.B, a.k_tok, C::TOKS, C::HB);
  if (e == cudaSuccess && a.k) e = make_tmap_f32_tokens(&m[4], dk, D, a.Hkv, a.L, a.B, C::TOKS, C::HB);
  if (e == cudaSuccess && dv) e = make_tmap_f32_tokens(&m[5], dv, D, a.Hkv, a.L, a.B, C::TOKS, C::HB);
  if (e != cudaSuccess) return e;
  if (!a.k) {  // not read
    m[1] = m[0];
    m[4] = m[3];
  }
  if (!dv) m[5] = m[3];
  m[2] = m[0];
  const int grid = staged_ctas<D, true, TPW>(p.list);
  e = staged_launch<D, true, TPW>(p, m, grid, s);
  if (e != cudaSuccess || (!dwq && !dwk)) return e;
  return launch_dependent(qk_rope_dw_kernel, dim3(2 * D / 32), dim3(1024), 0, s, p.part, dwq, dwk, D, grid);
}

}  // namespace

size_t qk_rope_bwd_part_floats(int D) { return (size_t)152 * 2 * 2 * D; }

cudaError_t launch_qk_rope_fwd(const RopeArgs& a, const uint16_t* v, long long v_tok, uint16_t* qo, uint16_t* ko,
                               uint16_t* vo, int kv_rows, int* status, cudaStream_t s) {
  StRope p = staged_params(a, v != nullptr, false, status);
  p.qo = qo;
  p.ko = ko;
  p.vo = vo;
  p.kv_rows = kv_rows;
  const bool few = tokens_a_warp(a, v != nullptr, false) == 4;
  switch (a.D) {
    case 64: return few ? staged_fwd<64, 4>(a, v, v_tok, p, s) : staged_fwd<64, 1>(a, v, v_tok, p, s);
    case 128: return few ? staged_fwd<128, 4>(a, v, v_tok, p, s) : staged_fwd<128, 1>(a, v, v_tok, p, s);
    case 256: return staged_fwd<256, 1>(a, v, v_tok, p, s);
    case 512: return staged_fwd<512, 1>(a, v, v_tok, p, s);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_qk_rope_bwd(const RopeArgs& a, const float* dq, const float* dk, const float* dv, uint16_t* gq,
                               uint16_t* gk, uint16_t* gv, long long gq_tok, long long gk_tok, long long gv_tok,
                               float* dwq, float* dwk, float* part, int* status, cudaStream_t s) {
  StRope p = staged_params(a, dv != nullptr, true, status);
  p.gq = gq;
  p.gk = gk;
  p.gv = gv;
  p.gq_tok = gq_tok;
  p.gk_tok = gk_tok;
  p.gv_tok = gv_tok;
  p.part = part;
  const bool few = tokens_a_warp(a, dv != nullptr, true) == 4;
  switch (a.D) {
    case 64: return few ? staged_bwd<64, 4>(a, dq, dk, dv, p, dwq, dwk, s) : staged_bwd<64, 1>(a, dq, dk, dv, p, dwq, dwk, s);
    case 128: return few ? staged_bwd<128, 4>(a, dq, dk, dv, p, dwq, dwk, s) : staged_bwd<128, 1>(a, dq, dk, dv, p, dwq, dwk, s);
    case 256: return staged_bwd<256, 1>(a, dq, dk, dv, p, dwq, dwk, s);
    case 512: return staged_bwd<512, 1>(a, dq, dk, dv, p, dwq, dwk, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace swa
