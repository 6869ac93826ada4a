// A cache in 8 bits: keys and values quantised as they are written, and read back.
//
// A cache holds e4m3 codes [B, Hkv, rows, D] and one fp32 scale for each block of
// 16 to 128 tokens of a head, [B, Hkv, ceil(rows / block)]; a value is code times
// scale.  The scale of a block is the smallest power of two s >= 2^-64 with
// max |x| <= 448 s over the block's tokens (448 is the largest e4m3 value): a
// floating code is as exact under a power of two as under max |x| / 448, and
// moving to a larger one is exact but for what falls below the smallest normal
// code, 2^-6 s.  So a block that has tokens keeps its scale while the new ones
// fit; otherwise its scale grows and its older codes are written again.
//
// Both kernels are bound by memory: an append reads 2 bytes and writes 1 an
// element, a read the other way round.  A group of threads has one block: it
// keeps the block's new rows in registers between the maximum and the codes, so
// they are read once.  Measured: 30,553 tokens of 16 heads, D = 256, appended in
// 110 us (6.8 TB/s), 2 x 16,384 rows of 4 heads, D = 512, half of them behind the
// lengths, read in 50.6 us (6.6 TB/s), one token of each of 64 requests appended in
// 1.8 us (2.5 us of the host's).  Blocks that keep another quantiser's scale divide
// (64 requests x 7 tokens of 8 heads, D = 256: 5.4 us, and 3.3 with powers of two).
//
// Maxima are those of bf16 patterns without their signs, two at a time: with fp32
// maxima and a division that no power of two needs the append was bound by its
// instructions (151 us).  A read's thread takes 8 codes, so that its 16 bytes and its
// neighbours' are written as whole lines (16 codes a thread: 59.5 us).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "cache8_rows.h"
#include "swa_internal.h"
#include "tc_ptx.cuh"

namespace swa {
namespace {

using namespace tc;

struct AppendParams {
  const uint16_t* x[2];      // k, v: bf16
  long long sb[2], sh[2], st[2];  // elements between requests, heads, tokens
  uint8_t* codes[2];
  float* scales[2];
  const int* kv_len;         // or null: tokens are rows 0 .. L - 1
  int B, Hkv, L, ld, rows, lb, nblk;  // ld, lb: log2 of D and of the block
  int nj;                    // blocks that a request's tokens meet at most
  int nx;                    // CTAs a head, or 0: groups go through all heads' blocks
};

// Four fp32 values to e4m3, nearest, 448 at most.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tcvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t codes) {  // the low two bytes
  uint32_t h;
  asm("{\n\t.reg .b16 lo;\n\tmov.b32 {lo, _}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(h) : "r"(codes));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
__device__ __forceinline__ float2 bf16x2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
// Pairs of bf16 patterns without their signs: as unsigned numbers they are in the order of the magnitudes.
__device__ __forceinline__ uint32_t magnitudes(uint32_t w) { return w & 0x7FFF7FFFu; }

// One block's new tokens by a group of GT threads, up to VPT vectors of 8
// elements each; MORE: rows behind those are read twice, for the maximum and, from
// L2, for the codes.
template <int GT, int VPT, bool MORE>
__global__ void __launch_bounds__(GT > 256 ? GT : 256, GT > 256 ? 2 : (VPT > 4 ? 3 : 6)) append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int CTA = GT > 256 ? GT : 256, GROUPS = CTA / GT;
  __shared__ uint32_t top[CTA / 32];
  grid_dependency_wait();
  grid_launch_dependents();
  const int which = blockIdx.y, group = threadIdx.x / GT, cta = blockIdx.x, tid = threadIdx.x % GT;
  // a CTA's groups have blocks of one head where there are as many (the quotients
  // are then the same for all threads, and formed once), or of neighbouring heads
  int bh, j;
  if (p.nx > 0) {
    bh = cta / p.nx;
    j = (cta - bh * p.nx) * GROUPS + group;
  } else {
    const int task = cta * GROUPS + group;
    bh = task / p.nj;
    j = task - bh * p.nj;
  }
  const bool in = j < p.nj && bh < p.B * p.Hkv;
  const int b = in ? bh / p.Hkv : 0, h = in ? bh - b * p.Hkv : 0;
  const int n = in ? (p.kv_len ? p.kv_len[b] : p.L) : 0;
  const Cache8Rows r = cache8_rows(n, p.L, p.rows, p.lb, j);
  const int blk = r.blk, lo = r.lo, a = r.a;
  const bool any = in && r.any;
  const int lv = p.ld - 3, vecs = any ? (r.hi - a) << lv : 0;  // vectors of the new rows
  const uint16_t* x = p.x[which] + b * p.sb[which] + h * p.sh[which] + r.token * p.st[which];
  auto vector = [&](int e) { return x + (e >> lv) * p.st[which] + ((e & ((1 << lv) - 1)) << 3); };
  uint32_t most = 0;  // the larger magnitude of a pair
  auto look = [&](const uint4& u) {
    most = __vmaxu2(most, __vmaxu2(magnitudes(u.x), magnitudes(u.y)));
    most = __vmaxu2(most, __vmaxu2(magnitudes(u.z), magnitudes(u.w)));
  };
  if (MORE) {
#pragma unroll 8
    for (int e = tid + VPT * GT; e < vecs; e += GT) look(*reinterpret_cast<const uint4*>(vector(e)));
  }
  uint4 v[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int e = tid + i * GT;
    v[i] = make_uint4(0, 0, 0, 0);
    // (a step is whole rows, but for 32 threads and rows of 512)
    const uint16_t* at = GT >= 64 || p.ld < 9 ? vector(tid) + i * ((GT >> lv) * p.st[which]) : vector(e);
    if (e < vecs) v[i] = __ldcs(reinterpret_cast<const uint4*>(at));
  }
  float* scale = p.scales[which] + (size_t)bh * p.nblk + blk;
  const bool older = any && a > lo;
  const float was = older ? *scale : 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) look(v[i]);
  most = max(most & 0xFFFFu, most >> 16);
  most = __reduce_max_sync(0xffffffffu, most);
  if (GT > 32) {
    if ((threadIdx.x & 31) == 0) top[threadIdx.x / 32] = most;
    __syncthreads();  // (also orders every thread's read of the old scale before it is written)
#pragma unroll
    for (int i = 0; i < GT / 32; ++i) most = max(most, top[group * (GT / 32) + i]);
  } else {
    __syncwarp();  // the same order within a warp: the reduction orders no memory
  }
  if (!any) return;
  const float amax = __uint_as_float(min(most, 0x7F7Fu) << 16);  // (infinity and NaN count as the largest number)
  const bool keep = older && amax <= 448.f * was;
  const float now = keep ? was : cache8_two_to(cache8_scale_exponent(amax, kCache8LeastExponent));
  uint8_t* codes = p.codes[which] + (((size_t)bh * p.rows) << p.ld);
  uint2* out = reinterpret_cast<uint2*>(codes + ((size_t)a << p.ld)) + tid;
  if ((__float_as_uint(now) & 0x7FFFFFu) == 0) {  // a power of two: its inverse is exact
    const uint64_t mul2 = f2_pack(1.f / now, 1.f / now);
    auto times = [&](uint32_t w) {
      const float2 f = bf16x2(w);
      return f2_unpack(f2_mul(f2_pack(f.x, f.y), mul2));
    };
    auto quantised = [&](const uint4& u) {
      const float2 x0 = times(u.x), x1 = times(u.y), x2 = times(u.z), x3 = times(u.w);
      return make_uint2(e4m3x4(x0.x, x0.y, x1.x, x1.y), e4m3x4(x2.x, x2.y, x3.x, x3.y));
    };
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (tid + i * GT < vecs) out[i * GT] = quantised(v[i]);
    if (MORE) {
#pragma unroll 8
      for (int e = tid + VPT * GT; e < vecs; e += GT) out[e - tid] = quantised(__ldcs(reinterpret_cast<const uint4*>(vector(e))));
    }
  } else {  // another quantiser's
#pragma unroll 1
    for (int e = tid; e < vecs; e += GT) {
      const uint4 u = *reinterpret_cast<const uint4*>(vector(e));
      const float2 x0 = bf16x2(u.x), x1 = bf16x2(u.y), x2 = bf16x2(u.z), x3 = bf16x2(u.w);
      out[e - tid] = make_uint2(e4m3x4(x0.x / now, x0.y / now, x1.x / now, x1.y / now),
                                e4m3x4(x2.x / now, x2.y / now, x3.x / now, x3.y / now));
    }
  }
  if (keep) return;
  if (tid == 0) *scale = now;
  if (older) {  // the older codes move to the new scale
    uint2* c = reinterpret_cast<uint2*>(codes + ((size_t)lo << p.ld));
    const int old = (a - lo) << lv;
    const float f = was / now;
#pragma unroll 1
    for (int e = tid; e < old; e += GT) {
      const uint2 u = c[e];
      const float2 x0 = from_e4m3x2(u.x), x1 = from_e4m3x2(u.x >> 16), x2 = from_e4m3x2(u.y), x3 = from_e4m3x2(u.y >> 16);
      c[e] = make_uint2(e4m3x4(x0.x * f, x0.y * f, x1.x * f, x1.y * f), e4m3x4(x2.x * f, x2.y * f, x3.x * f, x3.y * f));
    }
  }
}

struct ReadParams {
  const uint8_t* codes[2];
  const float* scales[2];
  uint16_t* out[2];
  const int* kv_len;  // or null: all rows
  int Hkv, ld, rows, lb, nblk;
  int row0, nrows;    // rows row0 .. row0 + nrows - 1 are read
  int nx;             // CTAs a head
};

constexpr int kReadThr = 256, kReadVec = 4;  // vectors of 8 codes a thread

__global__ void __launch_bounds__(kReadThr) read_kernel(const __grid_constant__ ReadParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int which = blockIdx.y, bh = blockIdx.x / p.nx, i = blockIdx.x - bh * p.nx;
  const int len = p.kv_len ? min(p.kv_len[bh / p.Hkv], p.rows) : p.rows;
  const int lv = p.ld - 3;
  const long long total = (long long)p.nrows << lv, e0 = (long long)i * kReadVec * kReadThr + threadIdx.x;  // vectors of a head
  const uint2* in = reinterpret_cast<const uint2*>(p.codes[which]) + (((size_t)bh * p.rows + p.row0) << lv) + e0;
  uint4* out = reinterpret_cast<uint4*>(p.out[which]) + (((size_t)bh * p.nrows) << lv) + e0;
  const float* scales = p.scales[which] + (size_t)bh * p.nblk;
  uint2 v[kReadVec];
  float s[kReadVec];
#pragma unroll
  for (int k = 0; k < kReadVec; ++k) {
    const long long e = e0 + k * kReadThr;
    const int row = p.row0 + (int)(e >> lv);
    v[k] = make_uint2(0, 0);
    s[k] = 0.f;
    if (e < total && row < len) {
      v[k] = __ldcs(in + k * kReadThr);
      s[k] = scales[row >> p.lb];
    }
  }
#pragma unroll
  for (int k = 0; k < kReadVec; ++k) {
    if (e0 + k * kReadThr >= total) return;
    const uint32_t w[4] = {v[k].x, v[k].x >> 16, v[k].y, v[k].y >> 16};
    uint32_t r[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float2 f = from_e4m3x2(w[q]);
      const __nv_bfloat162 o = __floats2bfloat162_rn(f.x * s[k], f.y * s[k]);
      r[q] = *reinterpret_cast<const uint32_t*>(&o);
    }
    out[k * kReadThr] = make_uint4(r[0], r[1], r[2], r[3]);
  }
}

int log2_of(int x) {
  int l = 0;
  while ((1 << l) < x) ++l;
  return l;
}

template <int GT, int VPT, bool MORE = false>
cudaError_t append_as(AppendParams& p, int tensors, cudaStream_t st) {
  constexpr int CTA = GT > 256 ? GT : 256, GROUPS = CTA / GT;
  const long long heads = (long long)p.B * p.Hkv;
  p.nx = p.nj >= GROUPS ? (p.nj + GROUPS - 1) / GROUPS : 0;
  const long long ctas = p.nx ? heads * p.nx : (heads * p.nj + GROUPS - 1) / GROUPS;
  return launch_dependent(append_kernel<GT, VPT, MORE>, dim3((unsigned)ctas, (unsigned)tensors), dim3(CTA), 0, st, p);
}

}  // namespace

cudaError_t launch_cache8_append(const Cache8AppendArgs& a, cudaStream_t st) {
  AppendParams p;
  int tensors = 0;
  for (int i = 0; i < 2; ++i) {
    if (!a.x[i]) continue;
    p.x[tensors] = a.x[i];
    p.sb[tensors] = a.stride_b[i];
    p.sh[tensors] = a.stride_h[i];
    p.st[tensors] = a.stride_t[i];
    p.codes[tensors] = a.codes[i];
    p.scales[tensors] = a.scales[i];
    ++tensors;
  }
  for (int i = tensors; i < 2; ++i) {
    p.x[i] = nullptr;
    p.codes[i] = nullptr;
    p.scales[i] = nullptr;
    p.sb[i] = p.sh[i] = p.st[i] = 0;
  }
  p.kv_len = a.kv_len;
  p.B = a.B;
  p.Hkv = a.Hkv;
  p.L = a.L;
  p.ld = log2_of(a.D);
  p.rows = a.rows;
  p.lb = log2_of(a.block);
  p.nblk = (a.rows + a.block - 1) / a.block;
  const long long meets = ((long long)a.L + a.block - 2) / a.block + 1;
  p.nj = (int)(meets < p.nblk ? meets : p.nblk);
  // the smallest group whose registers hold the new rows that a block can get: 8
  // vectors a thread (4 of 256 threads are as fast and more of a short prompt's loads
  // are under way at once; in smaller groups they are not: 4.8 TB/s and 6.4, for what
  // a thread does for its block weighs more), 2 of a step's few
  const long long vecs = (long long)(a.L < a.block ? a.L : a.block) * a.D / 8;
  if (vecs <= 32 * 2) return append_as<32, 2>(p, tensors, st);
  if (vecs <= 32 * 4) return append_as<32, 4>(p, tensors, st);
  if (vecs <= 32 * 8) return append_as<32, 8>(p, tensors, st);
  if (vecs <= 64 * 8) return append_as<64, 8>(p, tensors, st);
  if (vecs <= 256 * 4) return append_as<256, 4>(p, tensors, st);
  if (vecs <= 256 * 8) return append_as<256, 8>(p, tensors, st);
  if (vecs <= 512 * 8) return append_as<512, 8>(p, tensors, st);
  return append_as<512, 8, true>(p, tensors, st);  // 128 rows of 512: half of them once more from L2
}

cudaError_t launch_cache8_read(const Cache8ReadArgs& a, cudaStream_t st) {
  ReadParams p;
  int tensors = 0;
  for (int i = 0; i < 2; ++i) {
    if (!a.codes[i]) continue;
    p.codes[tensors] = a.codes[i];
    p.scales[tensors] = a.scales[i];
    p.out[tensors] = a.out[i];
    ++tensors;
  }
  for (int i = tensors; i < 2; ++i) {
    p.codes[i] = nullptr;
    p.scales[i] = nullptr;
    p.out[i] = nullptr;
  }
  p.kv_len = a.kv_len;
  p.Hkv = a.Hkv;
  p.ld = log2_of(a.D);
  p.rows = a.rows;
  p.lb = log2_of(a.block);
  p.nblk = (a.rows + a.block - 1) / a.block;
  p.row0 = a.row0;
  p.nrows = a.nrows;
  const long long per = (long long)kReadThr * kReadVec;
  p.nx = (int)((((long long)a.nrows * a.D / 8) + per - 1) / per);
  return launch_dependent(read_kernel, dim3((unsigned)((long long)a.B * a.Hkv * p.nx), (unsigned)tensors),
                          dim3(kReadThr), 0, st, p);
}

}  // namespace swa
