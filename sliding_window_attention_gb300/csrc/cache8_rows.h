// Which rows of a cache in scale blocks an append writes: plain arithmetic,
// without CUDA headers, so that it is checked on the host as well.
#pragma once

#ifdef __CUDACC__
#define SWA_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define SWA_HOST_DEVICE inline
#endif

namespace swa {

struct Cache8Rows {
  int blk;        // the block
  bool any;       // whether it gets a token
  int lo, a, hi;  // if so: its older tokens are rows lo .. a - 1, its new ones a .. hi - 1
  int token;      // and row a gets this one
};

// The j-th block that L tokens, the last of a request's first n rows, may meet
// in a cache of `rows` rows and blocks of 2^lb.  n is any int; 1 <= L, 1 <= rows <=
// 2e9, and j is below the cache's number of blocks.  Numbers of rows are unsigned, and a
// request that ends behind the cache begins at its end at most, so that none
// passes 2 * 2e9 + 256 < 2^32.
SWA_HOST_DEVICE Cache8Rows cache8_rows(int n, int L, int rows, int lb, int j) {
  const int from = n > L ? n - L : 0;  // row of token 0, or of the first that is not before the cache
  const unsigned row0 = (unsigned)(from < rows ? from : rows);
  const unsigned blk = (row0 >> lb) + (unsigned)j, lo = blk << lb, end = lo + (1u << lb);
  const unsigned a = lo > row0 ? lo : row0, top = (unsigned)(n < 0 ? 0 : (n < rows ? n : rows));
  const unsigned hi = end < top ? end : top;
  Cache8Rows r;
  r.any = a < hi;
  r.blk = r.any ? (int)blk : 0;
  r.lo = r.any ? (int)lo : 0;
  r.a = r.any ? (int)a : 0;
  r.hi = r.any ? (int)hi : 0;
  r.token = r.any ? (int)a - (n - L) : 0;
  return r;
}

}  // namespace swa
