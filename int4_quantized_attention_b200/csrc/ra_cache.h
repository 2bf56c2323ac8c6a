// ra_cache.h -- problem and launch interface of the paged cache's page
// operations (ra_cache.cu), shared with the C ABI (ra_serve_api.cu).
#pragma once
#include "ra_internal.h"

namespace ra {

struct CacheProb {
  int layers, n_pages, page_size, page_shift, Hkv, max_seqs, max_pages;
  uint8_t *k, *v;               // [layers][n_pages][Hkv][page_size][256 bytes]
  int *refs, *lens, *table;
};

// Workspace of the page operations (after the 256-byte header).
struct CacheWs {
  size_t jobs, mark, held, rank, list, map, src, dst, rows, total;
};
inline CacheWs cache_ws(int n_pages, int max_seqs) {
  CacheWs L;
  size_t o = align256(sizeof(WsHeader));
  const size_t pages = align256(sizeof(int) * (size_t)n_pages), seqs = align256(sizeof(int) * (size_t)max_seqs);
  const size_t most = pages > seqs ? pages : seqs;   // a fork has a job per child, a compaction one per page
  L.jobs = o;
  o += 256;
  L.mark = o;
  o += seqs;
  L.held = o;
  o += seqs;
  L.rank = o;
  o += seqs;
  L.list = o;
  o += pages;
  L.map = o;
  o += pages;
  L.src = o;
  o += most;
  L.dst = o;
  o += most;
  L.rows = o;
  o += most;
  L.total = o;
  return L;
}

cudaError_t launch_cache_extend(const CacheProb& c, const int* seqs, const int* n_new, int n, void* ws,
                                cudaStream_t st);
cudaError_t launch_cache_fork(const CacheProb& c, const int* parents, const int* children, int n, void* ws,
                              cudaStream_t st);
cudaError_t launch_cache_free(const CacheProb& c, const int* seqs, int n, void* ws, cudaStream_t st);
cudaError_t launch_cache_compact(const CacheProb& c, void* ws, cudaStream_t st);
cudaError_t launch_cache_write(const CacheProb& c, int layer, const int* seqs, const int* cu_new, int n, int total,
                               const uint8_t* k, const uint8_t* v, long long k_tok, long long k_head, long long v_tok,
                               long long v_head, void* ws, cudaStream_t st);

}  // namespace ra
