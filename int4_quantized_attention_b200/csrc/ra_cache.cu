// ra_cache.cu -- the pages of a key/value cache: giving pages to sequences
// that grow, writing new tokens into them, sharing them between sequences
// (fork), returning them (free) and moving the live ones together (compact).
//
// State: refs[page] = number of table entries that name the page (0: free),
// lens[row] = tokens of the sequence in that row, table[row][0 .. ceil(len /
// page_size)) = its pages, -1 behind them.  All of it is device memory and
// changes in stream order, so a captured graph may hold these calls.
//   - A page is given out lowest number first, in the order of the call's list.
//   - A part-filled last page belongs to one sequence alone: fork shares the
//     full pages and copies the filled tokens of the last one.
//   - compact: with n live pages, the i-th free page below n takes the
//     contents of the i-th live page at or above n, so as few pages move as
//     can, and no page is read after it was written.
//
// The state part of each call runs on one cluster of 8 CTAs, whose barrier
// orders its steps (check everything, then change; a call that cannot be
// carried out changes nothing and reports why).  Counting pages is the only
// step over all of refs: 4 bytes per page.  The bytes themselves are moved by
// copy_kernel over the whole GPU from a list of (source, destination, tokens).
// A write changes no state; it too is checked as a whole before it stores.
// A step's results depend on the lists and on prefix sums only, not on the
// order in which threads get there.
#include <cstdint>

#include "ra_cache.h"
#include "ra_launch.cuh"

namespace ra {
namespace {

constexpr int CL = 8;              // CTAs of the state cluster
constexpr int CT = 1024;           // threads per CTA of it
constexpr int ALL = CL * CT;
constexpr int COPY_CTAS = 8 * 148;   // 2048 threads per SM
constexpr int WRITE_CT = 256;      // threads per CTA of a write

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ int ctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return (int)r;
}
__device__ __forceinline__ int read_peer(const int* p, int rank) {
  uint32_t a;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

struct Sums {
  int need, pages, flags;
};
struct Shared {
  int need[32], pages[32], flags[32];   // per warp
  Sums total;                           // this CTA's
};

// Of every thread's `need` and `pages` the exclusive prefix over the cluster's
// threads (in thread order of CTA 0, 1, ...), all of them together, and the
// OR of the flags.  Every thread of the cluster calls it; one exchange for all
// three, since what a state call costs are its cluster barriers.
struct Scan {
  Sums before, all;
};
__device__ Scan cluster_scan(int need, int pages, int flags, Shared* sh) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int a = need, b = pages;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, a, d), y = __shfl_up_sync(0xffffffffu, b, d);
    if (lane >= d) a += x, b += y;
  }
  flags = __reduce_or_sync(0xffffffffu, flags);
  if (lane == 31) sh->need[warp] = a, sh->pages[warp] = b, sh->flags[warp] = flags;
  __syncthreads();
  if (warp == 0) {
    const int v = sh->need[lane], w = sh->pages[lane], f = __reduce_or_sync(0xffffffffu, sh->flags[lane]);
    int x = v, y = w;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int p = __shfl_up_sync(0xffffffffu, x, d), q = __shfl_up_sync(0xffffffffu, y, d);
      if (lane >= d) x += p, y += q;
    }
    sh->need[lane] = x - v;
    sh->pages[lane] = y - w;
    if (lane == 31) sh->total = {x, y, f};
  }
  cluster_barrier();
  Scan r{};
#pragma unroll
  for (int c = 0; c < CL; ++c) {
    const int x = read_peer(&sh->total.need, c), y = read_peer(&sh->total.pages, c);
    r.all.flags |= read_peer(&sh->total.flags, c);
    if (c < ctarank()) r.before.need += x, r.before.pages += y;
    r.all.need += x;
    r.all.pages += y;
  }
  r.before.need += sh->need[warp] + a - need;
  r.before.pages += sh->pages[warp] + b - pages;
  cluster_barrier();   // no CTA reuses its sums, nor ends, before every peer has read them
  return r;
}

struct Ws {
  WsHeader* hdr;
  int *jobs, *mark, *held, *rank, *list, *map, *src, *dst, *rows;
};
__host__ Ws ws_of(const CacheProb& c, void* ws) {
  const CacheWs L = cache_ws(c.n_pages, c.max_seqs);
  char* b = static_cast<char*>(ws);
  auto at = [&](size_t o) { return reinterpret_cast<int*>(b + o); };
  return {static_cast<WsHeader*>(ws), at(L.jobs), at(L.mark), at(L.held), at(L.rank), at(L.list), at(L.map), at(L.src),
          at(L.dst), at(L.rows)};
}

__device__ __forceinline__ int pages_for(const CacheProb& c, int len) { return (len + c.page_size - 1) >> c.page_shift; }
__device__ __forceinline__ bool row_ok(const CacheProb& c, int row) {
  return row >= 0 && row < c.max_seqs && row_fits(c.lens[row], c.max_pages, c.page_shift);
}

enum : int { BAD = 1, TOO_MUCH = 2 };   // flags of a scan

// Marks the rows of a list: rows named twice, or by both lists of a fork, are
// found by the count.  -1 entries take no part.  Returns BAD or 0, by thread.
__device__ int check_rows(const CacheProb& c, const Ws& w, const int* rows, int n, const int* others) {
  const int at = ctarank() * CT + threadIdx.x;
  for (int i = at; i < n; i += ALL) {
    if (rows[i] >= 0 && rows[i] < c.max_seqs) w.mark[rows[i]] = 0;
    if (others != nullptr && others[i] >= 0 && others[i] < c.max_seqs) w.mark[others[i]] = 0;
  }
  cluster_barrier();
  int bad = 0;
  for (int i = at; i < n; i += ALL) {
    if (rows[i] == -1) continue;
    if (!row_ok(c, rows[i])) bad = BAD;
    else if (atomicAdd(&w.mark[rows[i]], 1) != 0) bad = BAD;
  }
  if (others != nullptr) {
    cluster_barrier();
    for (int i = at; i < n; i += ALL) {
      if (rows[i] == -1) continue;
      if (!row_ok(c, others[i]) || w.mark[others[i]] != 0) bad = BAD;
    }
  }
  return bad;
}

// This thread's run of pages (consecutive, so that ranks ascend with numbers).
struct Run {
  int p0, p1;
};
__device__ __forceinline__ Run page_run(const CacheProb& c) {
  const int per = (c.n_pages + ALL - 1) / ALL, at = ctarank() * CT + threadIdx.x;
  return {min(c.n_pages, at * per), min(c.n_pages, at * per + per)};
}
__device__ __forceinline__ int count_free(const CacheProb& c, Run r) {
  int n = 0;
#pragma unroll 4
  for (int p = r.p0; p < r.p1; ++p) n += c.refs[p] == 0;
  return n;
}
// The first `want` free pages, lowest first, into w.list.
__device__ __forceinline__ void list_free(const CacheProb& c, const Ws& w, Run r, int rank, int want) {
  for (int p = r.p0; p < r.p1 && rank < want; ++p)
    if (c.refs[p] == 0 && in_bounds(rank >= 0 && rank < c.n_pages, &w.hdr->err, 0x5101)) w.list[rank++] = p;
}

__device__ __forceinline__ void report_once(WsHeader* h, uint32_t bit, uint32_t site) {
  if (ctarank() == 0 && threadIdx.x == 0) report(&h->err, bit, site);
}
// Whether a call has to be refused; says so.
__device__ __forceinline__ bool refused(const Scan& s, WsHeader* h, uint32_t site) {
  if (s.all.flags & BAD) report_once(h, DEVERR_BOUNDS, site);
  else if ((s.all.flags & TOO_MUCH) || s.all.need > s.all.pages) report_once(h, DEVERR_FULL, site + 1);
  else return false;
  return true;
}

// A write that follows a refused extend in the stream would find no slots of its
// own and store over the row's last tokens.  So a refused extend leaves the rows
// it named in w.held, and writes pass those over, until a call gives the row
// slots or empties it, or the error has been read.  w.held means something only
// while the error word has DEVERR_HELD, since its contents are unspecified before.
// Only extend sets that bit, behind all of its threads' reading it.
__device__ __forceinline__ bool holding(const Ws& w) { return (w.hdr->err.word & DEVERR_HELD) != 0; }
// All threads of the cluster, after a refusal; `already` as the call found it.
__device__ void hold_rows(const CacheProb& c, const Ws& w, const int* rows, int n, bool already) {
  const int at = ctarank() * CT + threadIdx.x;
  if (!already) {
    for (int r = at; r < c.max_seqs; r += ALL) w.held[r] = 0;
    cluster_barrier();
  }
  for (int i = at; i < n; i += ALL)
    if (rows[i] >= 0 && rows[i] < c.max_seqs) w.held[rows[i]] = 1;
  if (at == 0) atomicOr(&w.hdr->err.word, DEVERR_HELD);
}

__global__ void __cluster_dims__(CL, 1, 1) __launch_bounds__(CT)
    extend_kernel(CacheProb c, const int* __restrict__ seqs, const int* __restrict__ n_new, int n, Ws w) {
  __shared__ Shared sh;
  const bool held = holding(w);
  int flags = check_rows(c, w, seqs, n, nullptr);
  // entries in list order, a run of consecutive ones per thread
  const int per = (n + ALL - 1) / ALL, at = ctarank() * CT + threadIdx.x;
  const int i0 = min(n, at * per), i1 = min(n, i0 + per);
  int need = 0;
  for (int i = i0; i < i1; ++i) {
    if (seqs[i] == -1 || !row_ok(c, seqs[i])) continue;
    const int len = c.lens[seqs[i]], add = n_new[i];
    if (add < 0) flags |= BAD;
    else if ((long long)len + add > (long long)c.max_pages << c.page_shift) flags |= TOO_MUCH;
    else need += pages_for(c, len + add) - pages_for(c, len);   // over distinct rows: at most max_seqs x max_pages < 2^31
  }
  const Run run = page_run(c);
  const Scan s = cluster_scan(need, count_free(c, run), flags, &sh);
  if (refused(s, w.hdr, 0x5001)) return hold_rows(c, w, seqs, n, held);
  list_free(c, w, run, s.before.pages, s.all.need);
  int r = s.before.need;
  for (int i = i0; i < i1; ++i) {
    w.rank[i] = r;
    if (seqs[i] != -1) r += pages_for(c, c.lens[seqs[i]] + n_new[i]) - pages_for(c, c.lens[seqs[i]]);
  }
  cluster_barrier();
  const int lane = threadIdx.x & 31;
  for (int i = at >> 5; i < n; i += ALL / 32) {
    const int row = seqs[i];
    if (row == -1) continue;
    const int len = c.lens[row], have = pages_for(c, len), more = pages_for(c, len + n_new[i]) - have, first = w.rank[i];
    for (int k = lane; k < more; k += 32) {
      if (!in_bounds(first + k < c.n_pages && have + k < c.max_pages, &w.hdr->err, 0x5102)) continue;
      const int page = w.list[first + k];
      if (!in_bounds(page >= 0 && page < c.n_pages, &w.hdr->err, 0x5103)) continue;
      c.table[(long long)row * c.max_pages + have + k] = page;
      c.refs[page] = 1;
    }
    __syncwarp();
    if (lane == 0) {
      c.lens[row] = len + n_new[i];
      if (held) w.held[row] = 0;
    }
  }
}

__global__ void __cluster_dims__(CL, 1, 1) __launch_bounds__(CT)
    fork_kernel(CacheProb c, const int* __restrict__ parents, const int* __restrict__ children, int n, Ws w) {
  __shared__ Shared sh;
  const bool held = holding(w);
  int flags = check_rows(c, w, children, n, parents);
  const int per = (n + ALL - 1) / ALL, at = ctarank() * CT + threadIdx.x;
  if (at == 0) w.jobs[0] = 0;   // nothing to copy if this call is refused
  const int i0 = min(n, at * per), i1 = min(n, i0 + per);
  int need = 0;
  for (int i = i0; i < i1; ++i) {
    if (children[i] == -1 || !row_ok(c, children[i]) || !row_ok(c, parents[i])) continue;
    if (c.lens[children[i]] != 0) flags |= BAD;
    need += (c.lens[parents[i]] & (c.page_size - 1)) != 0;
  }
  const Run run = page_run(c);
  const Scan s = cluster_scan(need, count_free(c, run), flags, &sh);
  if (refused(s, w.hdr, 0x5011)) return;
  list_free(c, w, run, s.before.pages, s.all.need);
  int r = s.before.need;
  for (int i = i0; i < i1; ++i) {
    w.rank[i] = r;
    if (children[i] != -1) r += (c.lens[parents[i]] & (c.page_size - 1)) != 0;
  }
  cluster_barrier();
  const int lane = threadIdx.x & 31;
  for (int i = at >> 5; i < n; i += ALL / 32) {
    const int child = children[i];
    if (child == -1) continue;
    const int parent = parents[i], len = c.lens[parent], full = len >> c.page_shift, rest = len & (c.page_size - 1);
    const int* from = c.table + (long long)parent * c.max_pages;
    int* to = c.table + (long long)child * c.max_pages;
    for (int k = lane; k < full; k += 32) {
      if (!in_bounds(k < c.max_pages, &w.hdr->err, 0x5104)) continue;
      const int page = from[k];
      to[k] = page;
      if ((uint32_t)page < (uint32_t)c.n_pages) atomicAdd(&c.refs[page], 1);
      else report(&w.hdr->err, DEVERR_BOUNDS, 0x5014);
    }
    if (lane == 0) {
      if (rest != 0 && in_bounds(full < c.max_pages && w.rank[i] >= 0 && w.rank[i] < c.n_pages, &w.hdr->err, 0x5105)) {
        const int page = w.list[w.rank[i]], old = from[full];
        to[full] = page;
        c.refs[page] = 1;
        w.src[w.rank[i]] = old;
        w.dst[w.rank[i]] = page;
        w.rows[w.rank[i]] = rest;
        if ((uint32_t)old >= (uint32_t)c.n_pages) {
          w.src[w.rank[i]] = 0;
          w.rows[w.rank[i]] = 0;
          report(&w.hdr->err, DEVERR_BOUNDS, 0x5014);
        }
      }
      c.lens[child] = len;
      if (held) w.held[child] = 0;
    }
  }
  if (at == 0) w.jobs[0] = s.all.need;
}

__global__ void __cluster_dims__(CL, 1, 1) __launch_bounds__(CT)
    free_kernel(CacheProb c, const int* __restrict__ seqs, int n, Ws w) {
  __shared__ Shared sh;
  const bool held = holding(w);
  if (refused(cluster_scan(0, 0, check_rows(c, w, seqs, n, nullptr), &sh), w.hdr, 0x5021)) return;
  const int lane = threadIdx.x & 31, at = ctarank() * CT + threadIdx.x;
  for (int i = at >> 5; i < n; i += ALL / 32) {
    const int row = seqs[i];
    if (row == -1) continue;
    const int have = pages_for(c, c.lens[row]);
    int* t = c.table + (long long)row * c.max_pages;
    for (int k = lane; k < have; k += 32) {
      const int page = t[k];
      if ((uint32_t)page < (uint32_t)c.n_pages) atomicSub(&c.refs[page], 1);
      else report(&w.hdr->err, DEVERR_BOUNDS, 0x5022);
      t[k] = -1;
    }
    __syncwarp();
    if (lane == 0) {
      c.lens[row] = 0;
      if (held) w.held[row] = 0;
    }
  }
}

__global__ void __cluster_dims__(CL, 1, 1) __launch_bounds__(CT) compact_kernel(CacheProb c, Ws w) {
  __shared__ Shared sh;
  const int at = ctarank() * CT + threadIdx.x;
  const Run run = page_run(c);
  const int live = (run.p1 - run.p0) - count_free(c, run);
  // a row of unknown length could not follow its pages
  int flags = 0;
  for (int r = at; r < c.max_seqs; r += ALL)
    if (!row_ok(c, r)) flags = BAD;
  if (at == 0) w.jobs[0] = -1;
  const Scan first = cluster_scan(0, live, flags, &sh);
  if (refused(first, w.hdr, 0x5033)) return;
  const int total = first.all.pages;
  int holes = 0, movers = 0;
  for (int p = run.p0; p < run.p1; ++p) {
    const bool is = c.refs[p] != 0;
    holes += !is && p < total;
    movers += is && p >= total;
  }
  const Scan s = cluster_scan(holes, movers, 0, &sh);
  const int n = s.all.need;   // as many free pages below `total` as live ones above
  int h = s.before.need, m = s.before.pages;
  for (int p = run.p0; p < run.p1; ++p) {
    const bool is = c.refs[p] != 0;
    w.map[p] = p;
    if (!is && p < total && in_bounds(h >= 0 && h < c.n_pages, &w.hdr->err, 0x5106)) w.dst[h++] = p;
    if (is && p >= total && in_bounds(m >= 0 && m < c.n_pages, &w.hdr->err, 0x5107)) w.src[m++] = p;
  }
  cluster_barrier();
  for (int i = at; i < n; i += ALL) {
    const int from = w.src[i], to = w.dst[i];
    if (!in_bounds((uint32_t)from < (uint32_t)c.n_pages && (uint32_t)to < (uint32_t)c.n_pages, &w.hdr->err, 0x5108)) continue;
    w.map[from] = to;
    w.rows[i] = c.page_size;
    c.refs[to] = c.refs[from];
    c.refs[from] = 0;
  }
  if (at == 0) w.jobs[0] = n;
}

// Copies the listed pages' tokens in every layer and head: one warp per
// (page, layer, keys or values, head), a contiguous run of tokens x 256 bytes.
// Memory-bound: each byte is read once and written once; 8 loads of 16 bytes
// per lane are in flight before the first store.  1.28 GB moved (a compaction)
// take 410 us: 6.16 TB/s read and written, 0.94 of the measured copy.  With
// `remap`, the table's entries follow the map as well.
__global__ void __launch_bounds__(256) copy_kernel(CacheProb c, Ws w, int remap) {
  const int lane = threadIdx.x & 31;
  const long long warp = ((long long)blockIdx.x * 256 + threadIdx.x) >> 5, warps = (long long)gridDim.x * 8;
  if (remap && w.jobs[0] >= 0) {   // -1: the compaction was refused
    for (long long row = warp; row < c.max_seqs; row += warps) {
      if (!row_ok(c, (int)row)) continue;
      const int have = pages_for(c, c.lens[row]);
      int* t = c.table + row * c.max_pages;
      for (int k = lane; k < have; k += 32) {
        const int page = t[k];
        if ((uint32_t)page < (uint32_t)c.n_pages) t[k] = w.map[page];
        else report(&w.hdr->err, DEVERR_BOUNDS, 0x5031);
      }
    }
  }
  const int per = 2 * c.layers * c.Hkv;
  const long long runs = (long long)w.jobs[0] * per;
  const long long head_bytes = (long long)c.page_size * 256, page_bytes = head_bytes * c.Hkv;
  for (long long run = warp; run < runs; run += warps) {
    const int job = (int)(run / per), part = (int)(run % per);
    const int head = part % c.Hkv, layer = (part / c.Hkv) % c.layers;
    if (!in_bounds((uint32_t)w.src[job] < (uint32_t)c.n_pages && (uint32_t)w.dst[job] < (uint32_t)c.n_pages &&
                       w.rows[job] >= 0 && w.rows[job] <= c.page_size && layer < c.layers, &w.hdr->err, 0x5109))
      continue;
    uint8_t* pool = part / c.Hkv >= c.layers ? c.v : c.k;
    const long long base = (long long)layer * c.n_pages * page_bytes + head * head_bytes;
    const uint4* src = reinterpret_cast<const uint4*>(pool + base + w.src[job] * page_bytes) + lane;
    uint4* dst = reinterpret_cast<uint4*>(pool + base + w.dst[job] * page_bytes) + lane;
    const int chunks = w.rows[job] * 16;   // 16-byte pieces
    for (int o = 0; o < chunks; o += 256) {
      uint4 x[8];
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (o + 32 * q + lane < chunks) x[q] = __ldcs(src + o + 32 * q);
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (o + 32 * q + lane < chunks) __stcs(dst + o + 32 * q, x[q]);
    }
  }
}

// ---------------------------------------------------------------- write
// A write is checked as a whole before any of it is stored.  The checks need
// one thread for each entry of the list and for each page that the tokens lie
// in; `at` of `all` threads call this.  Rows named twice are found elsewhere.
// Returns BAD or 0, by thread.
__device__ int check_write(const CacheProb& c, const Ws& w, const int* seqs, const int* cu_new, int n, int total, int at,
                           int all) {
  const bool held = holding(w);
  int bad = 0;
  auto entry = [&](int i, int& row, int& count) {   // false: nothing of it is written
    row = seqs[i];
    count = 1;
    if (cu_new != nullptr) {
      const int a = cu_new[i], b = cu_new[i + 1];
      if (a < 0 || b < a || b > total) {
        bad = BAD;
        return false;
      }
      count = b - a;
    }
    if (row == -1) return false;
    if (held && row >= 0 && row < c.max_seqs && w.held[row] != 0) return false;
    if (!row_ok(c, row) || c.lens[row] < count) {
      bad = BAD;
      return false;
    }
    return count > 0;
  };
  // entry i has floor(cu_new[i] / page_size) + 2 i as its first page's number:
  // count tokens lie in at most floor(count / page_size) + 2 pages
  const long long pages = cu_new == nullptr ? n : (total >> c.page_shift) + 2ll * n;
  for (long long u = at; u < pages; u += all) {
    int i = (int)u, j = 0, row, count;
    if (cu_new != nullptr) {
      auto first = [&](int e) { return (cu_new[e] >> c.page_shift) + 2ll * e; };
      int lo = 0, hi = n - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first(mid) <= u) lo = mid; else hi = mid - 1;
      }
      i = lo;
      const long long past = u - first(i);
      if (past < 0) continue;
      j = (int)min(past, 1ll << 30);
    }
    if (!entry(i, row, count)) continue;
    const int len = c.lens[row], slot = ((len - count) >> c.page_shift) + j;
    if (slot > (len - 1) >> c.page_shift) continue;
    const int page = c.table[(long long)row * c.max_pages + slot];
    // a page that other rows share holds their tokens too
    if ((uint32_t)page >= (uint32_t)c.n_pages || c.refs[page] > 1) bad = BAD;
  }
  if (cu_new != nullptr) {   // entries without tokens or with bad offsets have no page of their own above
    int row, count;
    for (int i = at; i < n; i += all) entry(i, row, count);
  }
  return bad;
}

// Long lists and many tokens: one cluster checks, the copy waits for its word.
__global__ void __cluster_dims__(CL, 1, 1) __launch_bounds__(CT)
    write_check_kernel(CacheProb c, const int* __restrict__ seqs, const int* __restrict__ cu_new, int n, int total, Ws w) {
  __shared__ Shared sh;
  dependents_may_start();
  const int at = ctarank() * CT + threadIdx.x;
  const int flags = check_rows(c, w, seqs, n, nullptr) | check_write(c, w, seqs, cu_new, n, total, at, ALL);
  const bool no = refused(cluster_scan(0, 0, flags, &sh), w.hdr, 0x5041);
  if (at == 0) w.jobs[1] = !no;
}

// New tokens into their slots: 16 lanes per (token, head, keys or values).
// CHECKED: write_check_kernel's word decides, and the copies wait for it with
// their data in hand.  Otherwise the list is short, and a second half of every
// CTA checks all of it meanwhile (short_write says when): a launch more costs
// small writes what they take altogether.
template <bool CHECKED>
__global__ void __launch_bounds__(CHECKED ? WRITE_CT : 2 * WRITE_CT)
    write_kernel(CacheProb c, int layer, const int* __restrict__ seqs, const int* __restrict__ cu_new, int n, int total,
                 const uint8_t* __restrict__ k, const uint8_t* __restrict__ v, long long k_tok, long long k_head,
                 long long v_tok, long long v_head, Ws w) {
  __shared__ int rows[CHECKED ? 1 : WRITE_CT];
  int bad = 0;
  uint4 x = make_uint4(0, 0, 0, 0);
  uint4* dst = nullptr;
  if (!CHECKED && threadIdx.x >= WRITE_CT) {
    const int me = threadIdx.x - WRITE_CT, row = me < n ? seqs[me] : -1;
    rows[me] = row;
    bad = check_write(c, w, seqs, cu_new, n, total, me, WRITE_CT);
    asm volatile("bar.sync 1, %0;" ::"n"(WRITE_CT) : "memory");
    if (row != -1) {
#pragma unroll 8
      for (int j = 0; j < n; ++j)
        if (j != me && rows[j] == row) bad = BAD;
    }
  } else {
    // this thread's piece and its slot; whatever a bad list names is passed over, the checks find it
    const int lane16 = threadIdx.x & 15;
    const long long unit = ((long long)blockIdx.x * WRITE_CT + threadIdx.x) >> 4;
    const int per = 2 * c.Hkv;
    const bool held = holding(w);
    if (unit < (long long)total * per) {
      const int t = (int)(unit / per), part = (int)(unit % per), head = part % c.Hkv;
      const bool is_v = part >= c.Hkv;
      int i = t, first = t, last = t + 1;
      if (cu_new != nullptr) {
        int lo = 0, hi = n - 1;
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (cu_new[mid] <= t) lo = mid; else hi = mid - 1;
        }
        i = lo;
        first = cu_new[i];
        last = cu_new[i + 1];
      }
      const int row = seqs[i];
      if (first >= 0 && t >= first && t < last && row != -1 && row_ok(c, row) && c.lens[row] >= last - first) {
        const int pos = c.lens[row] - (last - t);
        const int page = c.table[(long long)row * c.max_pages + (pos >> c.page_shift)];
        if ((uint32_t)page < (uint32_t)c.n_pages && !(held && w.held[row] != 0)) {
          const long long slot = (((long long)layer * c.n_pages + page) * c.Hkv + head) * c.page_size + (pos & (c.page_size - 1));
          if (in_bounds(slot < (long long)c.layers * c.n_pages * c.Hkv * c.page_size && pos >> c.page_shift < c.max_pages,
                        &w.hdr->err, 0x510a)) {
            x = reinterpret_cast<const uint4*>(is_v ? v + t * v_tok + head * v_head : k + t * k_tok + head * k_head)[lane16];
            dst = reinterpret_cast<uint4*>((is_v ? c.v : c.k) + slot * 256) + lane16;
          }
        }
      }
    }
  }
  if constexpr (CHECKED) {
    wait_for_predecessor();
    if (w.jobs[1] == 0) return;
  } else if (__syncthreads_or(bad)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) report(&w.hdr->err, DEVERR_BOUNDS, 0x5041);
    return;
  }
  if (dst != nullptr) *dst = x;
}

// Each CTA checks the whole list itself while that is little work, which grows
// with the list and with the CTAs (tokens x heads).  In every CTA / by a launch
// of its own, 8 heads: 64 single tokens 3.2 / 6.1 us, 250 6.1 / 6.6, 64 x 8
// tokens 5.5 / 7.1, 64 x 16 9.0 / 7.7, 250 x 3 19.7 / 7.9, one row of 1024 5.0 /
// 7.4, measured before pages and held rows were looked at too, which adds 0.1 to
// 0.4 us.  (Without any check: 2.2, 2.3, 3.7, 4.2, 4.2 and 3.4 us.)
bool short_write(const CacheProb& c, int n, int total) {
  return n <= WRITE_CT && total <= 4 * WRITE_CT && (long long)n * total * c.Hkv < 1 << 19;
}

cudaError_t launch_copy(const CacheProb& c, const Ws& w, int remap, cudaStream_t st) {
  copy_kernel<<<COPY_CTAS, 256, 0, st>>>(c, w, remap);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_extend(const CacheProb& c, const int* seqs, const int* n_new, int n, void* ws,
                                cudaStream_t st) {
  extend_kernel<<<CL, CT, 0, st>>>(c, seqs, n_new, n, ws_of(c, ws));
  return cudaGetLastError();
}

cudaError_t launch_cache_fork(const CacheProb& c, const int* parents, const int* children, int n, void* ws,
                              cudaStream_t st) {
  const Ws w = ws_of(c, ws);
  fork_kernel<<<CL, CT, 0, st>>>(c, parents, children, n, w);
  cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? launch_copy(c, w, 0, st) : e;
}

cudaError_t launch_cache_free(const CacheProb& c, const int* seqs, int n, void* ws, cudaStream_t st) {
  free_kernel<<<CL, CT, 0, st>>>(c, seqs, n, ws_of(c, ws));
  return cudaGetLastError();
}

cudaError_t launch_cache_compact(const CacheProb& c, void* ws, cudaStream_t st) {
  const Ws w = ws_of(c, ws);
  compact_kernel<<<CL, CT, 0, st>>>(c, w);
  cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? launch_copy(c, w, 1, st) : e;
}

cudaError_t launch_cache_write(const CacheProb& c, int layer, const int* seqs, const int* cu_new, int n, int total,
                               const uint8_t* k, const uint8_t* v, long long k_tok, long long k_head, long long v_tok,
                               long long v_head, void* ws, cudaStream_t st) {
  const Ws w = ws_of(c, ws);
  const long long threads = (long long)total * 2 * c.Hkv * 16;
  const unsigned grid = (unsigned)((threads + WRITE_CT - 1) / WRITE_CT);
  if (short_write(c, n, total)) {
    write_kernel<false><<<grid > 0 ? grid : 1, 2 * WRITE_CT, 0, st>>>(c, layer, seqs, cu_new, n, total, k, v, k_tok, k_head,
                                                                  v_tok, v_head, w);
    return cudaGetLastError();
  }
  write_check_kernel<<<CL, CT, 0, st>>>(c, seqs, cu_new, n, total, w);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || grid == 0) return e;
  return launch_after(true, write_kernel<true>, grid, WRITE_CT, 0, st, c, layer, seqs, cu_new, n, total, k, v, k_tok,
                      k_head, v_tok, v_head, w);
}

}  // namespace ra
