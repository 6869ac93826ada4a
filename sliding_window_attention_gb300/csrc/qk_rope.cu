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
// position times that fraction, modulo 2^64, is the exact phase (integer
// multiplication wraps as angles do), and sincospif takes its top 32 bits.
//
// All sums, the norm and the rotation are fp32; the only rounding to fewer
// bits is the one of each output to bf16 (half a step, 2^-9 relative).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "swa_internal.h"

namespace swa {
namespace {

constexpr int kThr = 256, kWarps = kThr / 32;

// A row is held by LPR lanes, E elements each in NV vectors of 8 (16 bytes of
// bf16): vector j of lane l holds elements 256 j + 8 l ... + 7, so that every
// vector load of a warp is one contiguous run.
template <int D>
struct RowCfg {
  static constexpr int NV = D == 512 ? 2 : 1;
  static constexpr int E = 8 * NV;
  static constexpr int LPR = D / E;     // lanes of a row
  static constexpr int RPW = 32 / LPR;  // rows of a warp at once
};

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t bf_pack(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void unpack8(const uint4& v, float* x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf_lo(w[i]);
    x[2 * i + 1] = bf_hi(w[i]);
  }
}
__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(bf_pack(x[0], x[1]), bf_pack(x[2], x[3]), bf_pack(x[4], x[5]), bf_pack(x[6], x[7]));
}
template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
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

// cos / sin of T consecutive tokens from `tok0`, as cs[t * pairs + i].
__device__ __forceinline__ void fill_cs(const RopePos& a, long long tok0, int T, long long n_tok, int L,
                                        const uint64_t* step, float2* cs) {
  for (int idx = threadIdx.x; idx < T * a.pairs; idx += kThr) {
    const int t = idx / a.pairs, i = idx - t * a.pairs;
    const long long tok = tok0 + t;
    if (tok < n_tok) cs[idx] = turn_cs(token_pos(a, (int)(tok / L), (int)(tok % L), L), step[i]);
  }
}

// One lane's share of a token's rotation: y_e = c_e u_e + s_e u_partner(e).
template <int D, bool INTER>
struct LaneRot {
  using C = RowCfg<D>;
  float c[C::E], s[C::E];
  // half-split pairs: the lane (and vector) that holds each vector's partners
  int src[C::NV], srcv[C::NV];

  __device__ __forceinline__ void place(int lane, int pairs) {
    if (INTER) return;
#pragma unroll
    for (int j = 0; j < C::NV; ++j) {
      const int d = 256 * j + 8 * (lane % C::LPR);
      const int pd = d < pairs ? d + pairs : (d < 2 * pairs ? d - pairs : d);
      src[j] = (lane & ~(C::LPR - 1)) | ((pd % (C::LPR * 8)) >> 3);
      srcv[j] = C::NV > 1 ? pd / 256 : 0;
    }
  }
  __device__ __forceinline__ void load(const float2* cs, int lane, int pairs) {
#pragma unroll
    for (int j = 0; j < C::NV; ++j) {
      const int d = 256 * j + 8 * (lane % C::LPR);
      if (INTER) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool in = d + 2 * i < 2 * pairs;
          const float2 v = in ? cs[d / 2 + i] : make_float2(1.f, 0.f);
          c[8 * j + 2 * i] = c[8 * j + 2 * i + 1] = v.x;
          s[8 * j + 2 * i] = -v.y;
          s[8 * j + 2 * i + 1] = v.y;
        }
      } else {
        const bool lo = d < pairs, in = d < 2 * pairs;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 v = in ? cs[(lo ? d : d - pairs) + i] : make_float2(1.f, 0.f);
          c[8 * j + i] = v.x;
          s[8 * j + i] = lo ? -v.y : v.y;
        }
      }
    }
  }
  // The partners' values of one register array (as many words a vector as given).
  template <int W, typename T>
  __device__ __forceinline__ void partners(const T (&x)[W], T (&xp)[W], int pairs) const {
    constexpr int PV = W / C::NV;
    if (C::NV > 1 && 4 * pairs > D) {
      // a pair may span the two vectors (always, when the whole head is rotated)
      if (2 * pairs == D) {
#pragma unroll
        for (int i = 0; i < W; ++i) xp[i] = x[(i + PV) % W];
        return;
      }
#pragma unroll
      for (int j = 0; j < C::NV; ++j)
#pragma unroll
        for (int i = 0; i < PV; ++i) {
          const T a = __shfl_sync(0xffffffffu, x[i], src[j]), b = __shfl_sync(0xffffffffu, x[PV * (C::NV - 1) + i], src[j]);
          xp[PV * j + i] = srcv[j] ? b : a;
        }
      return;
    }
#pragma unroll
    for (int i = 0; i < PV; ++i) xp[i] = __shfl_sync(0xffffffffu, x[i], src[0]);
    if (C::NV > 1) {
#pragma unroll
      for (int i = PV; i < W; ++i) xp[i] = x[i];  // beyond the rotated part
    }
  }
};

struct RopeFwd {
  const uint16_t *q, *k, *v;             // token-major rows; k, v may be null
  long long q_tok, k_tok, v_tok;         // elements between tokens
  const float *wq, *wk;                  // [D] or null
  RopePos pos;
  uint16_t *qo, *ko, *vo;                // [B, Hq, L, D], [B, Hkv, kv_rows, D]
  int B, L, Hq, Hkv, kv_rows, T;         // T tokens a CTA (1, 2, 4 or 8)
  float eps, off;
};

// A warp takes one token and a share of its heads: the token's rotation
// stays in registers over all of them.  8 / T warps share a token.
template <int D, bool INTER>
__global__ void __launch_bounds__(kThr) qk_rope_fwd_kernel(const RopeFwd p) {
  using C = RowCfg<D>;
  constexpr int NV = C::NV, E = C::E, LPR = C::LPR, RPW = C::RPW, U = 4 / NV;  // U row groups in flight
  extern __shared__ uint64_t sm[];
  uint64_t* step = sm;
  float2* cs = reinterpret_cast<float2*>(sm + p.pos.pairs);
  const int pairs = p.pos.pairs, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long n_tok = (long long)p.B * p.L, tok0 = (long long)blockIdx.x * p.T;
  for (int i = threadIdx.x; i < pairs; i += kThr) step[i] = turn_step(p.pos.inv_freq[i]);
  __syncthreads();
  fill_cs(p.pos, tok0, p.T, n_tok, p.L, step, cs);
  __syncthreads();
  const int t = warp % p.T, share = warp / p.T, shares = kWarps / p.T;
  const long long tok = tok0 + t;
  if (tok >= n_tok) return;
  const int b = (int)(tok / p.L), l = (int)(tok % p.L);
  const int sub = lane / LPR, d0 = 8 * (lane % LPR);
  LaneRot<D, INTER> rot;
  rot.place(lane, pairs);

  const int kv_row = p.pos.kv_len ? p.pos.kv_len[b] - p.L + l : l;
  const bool kv_ok = kv_row >= 0 && kv_row < p.kv_rows;  // rows outside the cache are not written

  // rows of one kind (q or k)
  auto rows = [&](const uint16_t* x, const float* w, uint16_t* out, int H, long long head_stride, bool store) {
    float ca[E], sb[E];  // c_e w_e and s_e w_partner(e)
    rot.load(cs + t * pairs, lane, pairs);
    {
      float we[E], wp[E];
#pragma unroll
      for (int e = 0; e < E; ++e) we[e] = w ? w[256 * (e >> 3) + d0 + (e & 7)] + p.off : 1.f;
      if constexpr (INTER) {
#pragma unroll
        for (int e = 0; e < E; ++e) wp[e] = we[e ^ 1];
      } else {
        rot.partners(we, wp, pairs);
      }
#pragma unroll
      for (int e = 0; e < E; ++e) {
        ca[e] = rot.c[e] * we[e];
        sb[e] = rot.s[e] * wp[e];
      }
    }
    for (int h0 = share * RPW; h0 < H; h0 += U * shares * RPW) {
      uint4 raw[U][NV];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = h0 + u * shares * RPW + sub;
#pragma unroll
        for (int j = 0; j < NV; ++j)
          raw[u][j] = h < H ? __ldcs(reinterpret_cast<const uint4*>(x + (size_t)h * D + 256 * j + d0)) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = h0 + u * shares * RPW + sub;
        if (h0 + u * shares * RPW >= H) break;  // uniform over the warp
        float f[E], y[E];
        uint32_t words[4 * NV], other[4 * NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          unpack8(raw[u][j], f + 8 * j);
          words[4 * j] = raw[u][j].x;
          words[4 * j + 1] = raw[u][j].y;
          words[4 * j + 2] = raw[u][j].z;
          words[4 * j + 3] = raw[u][j].w;
        }
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) ss = fmaf(f[e], f[e], ss);
        const float r = rsqrtf(row_sum<LPR>(ss) * (1.f / D) + p.eps);
        if constexpr (INTER) {
#pragma unroll
          for (int e = 0; e < E; ++e) y[e] = r * fmaf(f[e], ca[e], f[e ^ 1] * sb[e]);
        } else {
          rot.partners(words, other, pairs);
#pragma unroll
          for (int i = 0; i < 4 * NV; ++i) {
            y[2 * i] = r * fmaf(f[2 * i], ca[2 * i], bf_lo(other[i]) * sb[2 * i]);
            y[2 * i + 1] = r * fmaf(f[2 * i + 1], ca[2 * i + 1], bf_hi(other[i]) * sb[2 * i + 1]);
          }
        }
        if (store && h < H) {
#pragma unroll
          for (int j = 0; j < NV; ++j)
            *reinterpret_cast<uint4*>(out + h * head_stride + 256 * j + d0) = pack8(y + 8 * j);
        }
      }
    }
  };
  rows(p.q + tok * p.q_tok, p.wq, p.qo + (((size_t)b * p.Hq) * p.L + l) * D, p.Hq, (long long)p.L * D, true);
  const size_t kv_off = ((size_t)b * p.Hkv * p.kv_rows + (kv_ok ? kv_row : 0)) * D;
  if (p.k) rows(p.k + tok * p.k_tok, p.wk, p.ko + kv_off, p.Hkv, (long long)p.kv_rows * D, kv_ok);
  if (p.v && kv_ok) {
    const uint16_t* x = p.v + tok * p.v_tok;
    for (int h = share * RPW + sub; h < p.Hkv; h += shares * RPW)
#pragma unroll
      for (int j = 0; j < NV; ++j)
        *reinterpret_cast<uint4*>(p.vo + kv_off + (size_t)h * p.kv_rows * D + 256 * j + d0) =
            __ldcs(reinterpret_cast<const uint4*>(x + (size_t)h * D + 256 * j + d0));
  }
}

struct RopeBwd {
  const uint16_t *q, *k;                 // the forward's inputs; k may be null
  long long q_tok, k_tok;
  const float *wq, *wk;                  // [D] or null
  RopePos pos;
  const float *dq, *dk, *dv;             // [B, H, L, D]; dk, dv may be null
  uint16_t *gq, *gk, *gv;                // gradient rows, token-major
  long long gq_tok, gk_tok, gv_tok;
  float* part;                           // [gridDim.x][2][D] partial dw
  int B, L, Hq, Hkv;
  float eps, off;
};

// Persistent: a CTA walks blocks of kWarps consecutive tokens, a warp a
// token; the scales' gradients stay in registers until the end and leave as
// one partial sum a CTA, so their order of summation is fixed by the launch.
template <int D, bool INTER>
__global__ void __launch_bounds__(kThr) qk_rope_bwd_kernel(const RopeBwd p) {
  using C = RowCfg<D>;
  constexpr int NV = C::NV, E = C::E, LPR = C::LPR, RPW = C::RPW;
  extern __shared__ uint64_t sm[];
  uint64_t* step = sm;
  float2* cs = reinterpret_cast<float2*>(sm + p.pos.pairs);
  const int pairs = p.pos.pairs, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long n_tok = (long long)p.B * p.L;
  const int sub = lane / LPR, d0 = 8 * (lane % LPR);
  for (int i = threadIdx.x; i < pairs; i += kThr) step[i] = turn_step(p.pos.inv_freq[i]);
  LaneRot<D, INTER> rot;
  rot.place(lane, pairs);
  float accq[E], acck[E];
#pragma unroll
  for (int e = 0; e < E; ++e) accq[e] = acck[e] = 0.f;

  for (long long tok0 = (long long)blockIdx.x * kWarps; tok0 < n_tok; tok0 += (long long)gridDim.x * kWarps) {
    __syncthreads();  // step[] is written; the last block's cs[] is consumed
    fill_cs(p.pos, tok0, kWarps, n_tok, p.L, step, cs);
    __syncthreads();
    const long long tok = tok0 + warp;
    if (tok >= n_tok) continue;
    const int b = (int)(tok / p.L), l = (int)(tok % p.L);
    rot.load(cs + warp * pairs, lane, pairs);

    auto rows = [&](const uint16_t* x, const float* w, const float* dy, uint16_t* out, int H, float (&acc)[E]) {
      float we[E];
#pragma unroll
      for (int e = 0; e < E; ++e) we[e] = w ? w[256 * (e >> 3) + d0 + (e & 7)] + p.off : 1.f;
#pragma unroll 2
      for (int hg = 0; hg < H; hg += RPW) {
        const int h = hg + sub;
        const bool in = h < H;
        float f[E], g[E], gp[E];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const uint4 raw = in ? __ldcs(reinterpret_cast<const uint4*>(x + (size_t)h * D + 256 * j + d0)) : make_uint4(0, 0, 0, 0);
          const float4* dyp = reinterpret_cast<const float4*>(dy + (size_t)h * p.L * D + 256 * j + d0);
          const float4 a = in ? __ldcs(dyp) : make_float4(0.f, 0.f, 0.f, 0.f);
          const float4 c = in ? __ldcs(dyp + 1) : make_float4(0.f, 0.f, 0.f, 0.f);
          unpack8(raw, f + 8 * j);
          g[8 * j] = a.x; g[8 * j + 1] = a.y; g[8 * j + 2] = a.z; g[8 * j + 3] = a.w;
          g[8 * j + 4] = c.x; g[8 * j + 5] = c.y; g[8 * j + 6] = c.z; g[8 * j + 7] = c.w;
        }
        // the rotation's transpose: c_e dy_e - s_e dy_partner(e)
        if constexpr (INTER) {
#pragma unroll
          for (int e = 0; e < E; ++e) gp[e] = g[e ^ 1];
        } else {
          rot.partners(g, gp, pairs);
        }
        float ss = 0.f, dot = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          g[e] = fmaf(rot.c[e], g[e], -rot.s[e] * gp[e]);
          ss = fmaf(f[e], f[e], ss);
          dot = fmaf(g[e] * we[e], f[e], dot);
        }
        ss = row_sum<LPR>(ss);
        dot = row_sum<LPR>(dot);
        const float r = rsqrtf(ss * (1.f / D) + p.eps);
        const float m = dot * r * r * (1.f / D);  // mean(h n) r
#pragma unroll
        for (int e = 0; e < E; ++e) {
          acc[e] = fmaf(g[e] * r, f[e], acc[e]);
          g[e] = r * (g[e] * we[e] - f[e] * m);
        }
        if (in) {
#pragma unroll
          for (int j = 0; j < NV; ++j) *reinterpret_cast<uint4*>(out + (size_t)h * D + 256 * j + d0) = pack8(g + 8 * j);
        }
      }
    };
    rows(p.q + tok * p.q_tok, p.wq, p.dq + ((size_t)b * p.Hq * p.L + l) * D, p.gq + tok * p.gq_tok, p.Hq, accq);
    if (p.k) rows(p.k + tok * p.k_tok, p.wk, p.dk + ((size_t)b * p.Hkv * p.L + l) * D, p.gk + tok * p.gk_tok, p.Hkv, acck);
    if (p.dv) {
      for (int h = sub; h < p.Hkv; h += RPW)
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const float4* dvp = reinterpret_cast<const float4*>(p.dv + (((size_t)b * p.Hkv + h) * p.L + l) * D + 256 * j + d0);
          const float4 a = __ldcs(dvp), c = __ldcs(dvp + 1);
          const float y[8] = {a.x, a.y, a.z, a.w, c.x, c.y, c.z, c.w};
          *reinterpret_cast<uint4*>(p.gv + tok * p.gv_tok + (size_t)h * D + 256 * j + d0) = pack8(y);
        }
    }
  }

  // this CTA's dw: the warp's row slots, then the warps, in a fixed order
  __syncthreads();
  float* red = reinterpret_cast<float*>(sm);  // [kWarps][D]
#pragma unroll
  for (int kind = 0; kind < 2; ++kind) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      float v = kind ? acck[e] : accq[e];
#pragma unroll
      for (int o = LPR; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (sub == 0) red[warp * D + 256 * (e >> 3) + d0 + (e & 7)] = v;
    }
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += kThr) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v += red[w * D + d];
      p.part[((size_t)blockIdx.x * 2 + kind) * D + d] = v;
    }
    __syncthreads();
  }
}

// dw[kind][d] = sum of the CTAs' partials, 8 strided sums a column, then those.
__global__ void __launch_bounds__(256) qk_rope_dw_kernel(const float* part, float* dwq, float* dwk, int D, int n) {
  __shared__ float red[8][32];
  const int col = blockIdx.x * 32 + (threadIdx.x & 31), grp = threadIdx.x >> 5;  // column of [2][D]
  float v = 0.f;
#pragma unroll 8
  for (int c = grp; c < n; c += 8) v += part[(size_t)c * 2 * D + col];
  red[grp][threadIdx.x & 31] = v;
  __syncthreads();
  if (grp == 0) {
#pragma unroll
    for (int g = 1; g < 8; ++g) v += red[g][threadIdx.x];
    float* out = col < D ? dwq : dwk;
    if (out) out[col < D ? col : col - D] = v;
  }
}

template <int D>
cudaError_t rope_fwd_d(const RopeFwd& p, cudaStream_t s) {
  const long long n_tok = (long long)p.B * p.L;
  const unsigned grid = (unsigned)((n_tok + p.T - 1) / p.T);
  const size_t smem = (size_t)p.pos.pairs * 8 * (1 + p.T);
  if (p.pos.interleaved) qk_rope_fwd_kernel<D, true><<<grid, kThr, smem, s>>>(p);
  else qk_rope_fwd_kernel<D, false><<<grid, kThr, smem, s>>>(p);
  return cudaGetLastError();
}

template <int D>
cudaError_t rope_bwd_d(const RopeBwd& p, int grid, float* dwq, float* dwk, cudaStream_t s) {
  const size_t cs = (size_t)p.pos.pairs * 8 * (1 + kWarps), red = (size_t)kWarps * D * 4;
  const size_t smem = cs > red ? cs : red;
  if (p.pos.interleaved) qk_rope_bwd_kernel<D, true><<<grid, kThr, smem, s>>>(p);
  else qk_rope_bwd_kernel<D, false><<<grid, kThr, smem, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || (!dwq && !dwk)) return e;
  qk_rope_dw_kernel<<<2 * D / 32, 256, 0, s>>>(p.part, dwq, dwk, D, grid);
  return cudaGetLastError();
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

constexpr int kBwdCtasPerSm = 2;

}  // namespace

int qk_rope_bwd_ctas(long long tokens) {
  const long long blocks = (tokens + kWarps - 1) / kWarps;
  return (int)(blocks < 152 * kBwdCtasPerSm ? blocks : 152 * kBwdCtasPerSm);
}

cudaError_t launch_qk_rope_fwd(const RopeArgs& a, const uint16_t* v, long long v_tok, uint16_t* qo, uint16_t* ko,
                               uint16_t* vo, int kv_rows, cudaStream_t s) {
  RopeFwd p;
  p.q = a.q;
  p.k = a.k;
  p.v = v;
  p.q_tok = a.q_tok;
  p.k_tok = a.k_tok;
  p.v_tok = v_tok;
  p.wq = a.wq;
  p.wk = a.wk;
  p.pos = rope_pos(a);
  p.qo = qo;
  p.ko = ko;
  p.vo = vo;
  p.B = a.B;
  p.L = a.L;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.kv_rows = kv_rows;
  p.eps = a.eps;
  p.off = a.weight_offset;
  const long long n_tok = (long long)a.B * a.L;
  p.T = n_tok >= 4096 ? 4 : 1;
  switch (a.D) {
    case 64: return rope_fwd_d<64>(p, s);
    case 128: return rope_fwd_d<128>(p, s);
    case 256: return rope_fwd_d<256>(p, s);
    case 512: return rope_fwd_d<512>(p, s);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_qk_rope_bwd(const RopeArgs& a, const float* dq, const float* dk, const float* dv, uint16_t* gq,
                               uint16_t* gk, uint16_t* gv, long long gq_tok, long long gk_tok, long long gv_tok,
                               float* dwq, float* dwk, float* part, cudaStream_t s) {
  RopeBwd p;
  p.q = a.q;
  p.k = a.k;
  p.q_tok = a.q_tok;
  p.k_tok = a.k_tok;
  p.wq = a.wq;
  p.wk = a.wk;
  p.pos = rope_pos(a);
  p.dq = dq;
  p.dk = dk;
  p.dv = dv;
  p.gq = gq;
  p.gk = gk;
  p.gv = gv;
  p.gq_tok = gq_tok;
  p.gk_tok = gk_tok;
  p.gv_tok = gv_tok;
  p.part = part;
  p.B = a.B;
  p.L = a.L;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.eps = a.eps;
  p.off = a.weight_offset;
  const int grid = qk_rope_bwd_ctas((long long)a.B * a.L);
  switch (a.D) {
    case 64: return rope_bwd_d<64>(p, grid, dwq, dwk, s);
    case 128: return rope_bwd_d<128>(p, grid, dwq, dwk, s);
    case 256: return rope_bwd_d<256>(p, grid, dwq, dwk, s);
    case 512: return rope_bwd_d<512>(p, grid, dwq, dwk, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace swa
