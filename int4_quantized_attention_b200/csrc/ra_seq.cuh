// ra_seq.cuh -- what the attention kernels over packed and paged sequences
// share: where a sequence lies, how its work is cut into shares, 16-bit types,
// where a row's result goes.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <atomic>
#include <cstdint>

#include "ra_launch.cuh"
#include "ra_serve.h"

namespace ra {

constexpr float LN2 = 0.6931471805599453f;
constexpr float RAISE = 8.0f;    // follow the row maximum when it rises by more than this (log2)
constexpr int NO_TILE = 0x7fffffff;

enum : int { OUT_FINAL = 0, OUT_SLOT = 1, OUT_LEAD = 2, OUT_OWN = 3 };

struct SeqInfo {
  int q0, Lq, k0, L, len, off, row;
};

// Sequence i's place; whatever the device-side inputs do not allow is
// reported and left out (Lq = 0 or L = 0).
__device__ __forceinline__ SeqInfo seq_info(const SeqProb& P, int i, DeviceErr* err) {
  SeqInfo s;
  s.row = -1;
  s.k0 = 0;
  s.L = 0;
  if (P.cu_q != nullptr) {
    s.q0 = P.cu_q[i];
    const int q1 = P.cu_q[i + 1];
    s.Lq = q1 - s.q0;
    if (s.q0 < 0 || q1 < s.q0 || q1 > P.total_q) {
      report(err, DEVERR_BOUNDS, 0x4001);
      s.q0 = 0;
      s.Lq = 0;
    }
  } else {
    s.q0 = i;
    s.Lq = 1;
  }
  if (P.paged) {
    const int r = P.seqs[i];
    if (r >= 0 && r < P.max_seqs) {
      const int L = P.lens[r];
      if (row_fits(L, P.max_pages, P.page_shift)) {
        s.row = r;
        s.L = L;
      } else {
        report(err, DEVERR_BOUNDS, 0x4002);
      }
    } else if (r != -1) {
      report(err, DEVERR_BOUNDS, 0x4003);
    }
  } else {
    const int k0 = P.cu_k[i], k1 = P.cu_k[i + 1];
    if (k0 < 0 || k1 < k0 || k1 > P.total_k) {
      report(err, DEVERR_BOUNDS, 0x4004);
    } else {
      s.k0 = k0;
      s.L = k1 - k0;
    }
  }
  s.len = s.L > P.shared ? s.L - P.shared : 0;
  s.off = s.L - s.Lq - P.shared;
  return s;
}

__host__ __device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }
// r / G for r < 128: the multiplier's error, at most r / 2^16, is below 1 / G.
__device__ __forceinline__ int over_G(const SeqProb& P, int r) { return (int)((uint32_t)r * P.inv_G >> 16); }
__device__ __forceinline__ int clampi(int x, int lo, int hi) { return min(max(x, lo), hi); }

// The sequence that token t belongs to: the largest i with cu_q[i] <= t.
__device__ __forceinline__ int seq_of_token(const SeqProb& P, int t) {
  if (P.cu_q == nullptr) return t;
  int lo = 0, hi = P.n_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (P.cu_q[mid] <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// ---------------------------------------------------------------- launches
// What a kernel needs set on each device before its first launch there (a
// device reset drops it, as it drops the caller's memory).
struct OncePerDevice {
  std::atomic<uint64_t> done{0};   // one bit per device; from the 64th on it is set every time
  template <class F>
  cudaError_t run(F set) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && (done.load(std::memory_order_acquire) >> dev & 1)) return cudaSuccess;
    e = set();
    if (e == cudaSuccess && dev < 64) done.fetch_or(1ull << dev, std::memory_order_release);
    return e;
  }
};

// ---------------------------------------------------------------- shares
// The two kernels a call may use.  KIND_MANY: 128-row query tiles on the
// tensor-memory MMA, items of two tiles.  KIND_FEW: at most FEW_ROWS rows over
// pages, one item per sequence and key head, on the warp-level MMA.
// All items are laid end to end, W_ITEM units for an item and one for each
// key it sees, and cut into one share per CTA.  A key tile goes to the CTA in
// whose share its first unit lies.
enum : int { KIND_MANY = 0, KIND_FEW = 1 };
template <int KIND>
struct Kind;
template <>
struct Kind<KIND_MANY> {
  static constexpr int TILE = KEYS, W_ITEM = 384, SLOT = SLOT_ROWS;
  __device__ static __forceinline__ int tokens_per_item(const SeqProb& P) { return 2 * P.TQ; }
};
template <>
struct Kind<KIND_FEW> {
  static constexpr int TILE = FEW_KEYS, W_ITEM = 160, SLOT = FEW_ROWS;
  __device__ static __forceinline__ int tokens_per_item(const SeqProb& P) { return FEW_ROWS; }
};

// Which kernel takes a sequence (or the shared region) with so many query tokens.
template <int KIND>
__device__ __forceinline__ bool takes(const SeqProb& P, int tokens) {
  return (P.paged && (long long)tokens * P.G <= FEW_ROWS) == (KIND == KIND_FEW);
}

// A row's place in its item's slot: token tt of the item, head gh of the group.
template <int KIND>
__device__ __forceinline__ int slot_row(const SeqProb& P, int tt, int gh) {
  return KIND == KIND_FEW ? tt * P.G + gh : (tt / P.TQ) * 128 + (tt % P.TQ) * P.G + gh;
}

// The items of one sequence's own region, or of the shared region: `count`
// per key head.  Item u sees span(u) keys (at least one is counted, so that
// rows without keys are written too); where the mask is causal that grows by
// `step` tokens from item to item.
template <int KIND>
struct Items {
  int count, base, step, tokens;
  __device__ __forceinline__ int span(int u) const {
    return max(1, base + (step ? (int)min((long long)(u + 1) * step, (long long)tokens) : 0));
  }
  __device__ __forceinline__ int tiles(int u) const { return ceil_div(span(u), Kind<KIND>::TILE); }
  // units before item u < count
  __device__ __forceinline__ long long before(int u) const {
    return (long long)u * (Kind<KIND>::W_ITEM + (step ? base : max(1, base))) + (long long)step * u * (u + 1) / 2;
  }
  __device__ __forceinline__ long long all() const {
    return count == 0 ? 0 : before(count - 1) + Kind<KIND>::W_ITEM + span(count - 1);
  }
};
template <int KIND>
__device__ __forceinline__ Items<KIND> items_of(const SeqProb& P, bool lead, const SeqInfo& s) {
  Items<KIND> i;
  i.tokens = lead ? P.total_q : s.Lq;
  const int per = Kind<KIND>::tokens_per_item(P);
  i.count = takes<KIND>(P, i.tokens) ? ceil_div(i.tokens, per) : 0;
  const bool grows = P.causal && !lead;
  i.base = lead ? P.shared : grows ? max(0, s.off) : s.len;
  i.step = grows ? per : 0;
  return i;
}

// a / b for a quotient that fits an int; mostly 32-bit.
__device__ __forceinline__ int quotient(long long a, long long b) {
  return (a | b) >> 32 == 0 ? (int)((uint32_t)a / (uint32_t)b) : (int)(a / b);
}

// A CTA's share of all units: more than a tile, so that every CTA between an
// item's first and last holds one of its tiles.
__device__ __forceinline__ long long share_of(long long total, int ctas) {
  const long long t = total + ctas - 1;
  return max(t >> 32 == 0 ? (long long)((uint32_t)t / (uint32_t)ctas) : t / ctas, 200ll);
}

// In shared memory: the plan of one CTA.
struct SharePlan {
  long long scan[16], best[16];
  long long total, first_start;
  int first_seq;             // sequence in which the share begins; -1: the shared region
  int lead_row, lead_len;    // the table row that the shared pages are read from, its length
};

// Lays all units end to end: the total, and where this CTA's share begins.
// All THREADS threads; ends with a barrier.  CTA 0 leaves the sequences'
// first units for the join.
template <int KIND, int THREADS>
__device__ void plan_shares(const SeqProb& P, SharePlan& plan, DeviceErr* err) {
  const ShareBuf& b = KIND == KIND_FEW ? P.few : P.many;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (KIND == KIND_MANY && P.lead_only) {
    // nothing depends on the lengths but whose pages are read: the first
    // sequence's, if it reaches so far (others do below)
    const SeqInfo first = seq_info(P, 0, nullptr);
    if (first.L >= P.shared) {
      if (tid == 0) {
        plan.total = items_of<KIND>(P, true, first).all() * P.Hkv;
        plan.first_seq = -1;
        plan.lead_row = first.row;
        plan.lead_len = first.L;
        if (blockIdx.x == 0) b.starts[P.n_seqs] = plan.total;
      }
      __syncthreads();
      return;
    }
  }
  const int per = ceil_div(P.n_seqs, THREADS);
  const int i0 = min(P.n_seqs, tid * per), i1 = min(P.n_seqs, i0 + per);
  long long sum = 0, best = -1;
  SeqInfo s{};
  for (int i = i0; i < i1; ++i) {
    s = seq_info(P, i, err);
    sum += items_of<KIND>(P, false, s).all() * P.Hkv;
    // the longest sequence, the first of them, gives the shared pages
    best = max(best, ((long long)s.L << 32) | (uint32_t)(0x7fffffff - i));
  }
  long long incl = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += x;
    if (P.shared > 0) best = max(best, __shfl_xor_sync(0xffffffffu, best, d));
  }
  if (lane == 31) plan.scan[warp] = incl;
  if (lane == 0) plan.best[warp] = best;
  if (tid == 0) plan.first_seq = -1;
  __syncthreads();
  const long long lead = P.shared > 0 ? items_of<KIND>(P, true, s).all() * P.Hkv : 0;
  long long total = lead, at = lead + incl - sum;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    const long long x = plan.scan[w];
    if (w < warp) at += x;
    total += x;
  }
  if (tid == 0) {
    plan.total = total;
    if (P.shared > 0) {
      for (int w = 1; w < THREADS / 32; ++w) best = max(best, plan.best[w]);
      const SeqInfo l = seq_info(P, 0x7fffffff - (int)(uint32_t)(best & 0xffffffffll), nullptr);
      plan.lead_row = l.row;
      plan.lead_len = l.L;
    }
    if (blockIdx.x == 0) b.starts[P.n_seqs] = total;
  }
  const long long mine = share_of(total, gridDim.x) * blockIdx.x;
  if (blockIdx.x == 0 || (mine >= at && mine < at + sum)) {
    for (int i = i0; i < i1; ++i) {
      if (per > 1) s = seq_info(P, i, nullptr);
      const long long n = items_of<KIND>(P, false, s).all() * P.Hkv;
      if (blockIdx.x == 0) b.starts[i] = at;
      if (mine >= at && mine < at + n) {
        plan.first_seq = i;
        plan.first_start = at;
      }
      at += n;
    }
  }
  __syncthreads();
}

template <int KIND>
struct ShareWalk {
  long long at, end;     // the share
  long long start;       // first unit of the next item
  int seq, kvh, u;       // sequence (-1: the shared region), key head and item of that
  int known;             // the sequence that `s` and `it` describe (-2: none)
  SeqInfo s;
  Items<KIND> it;
};
struct SharePart {
  int lead, tokens;      // the shared region?; the query tokens of the sequence (of all)
  int kvh, item;
  int t0, t1;            // key tiles
  int out, slot;
  int parts;             // OUT_SLOT, slot 1: the CTAs that the item is spread over
};

template <int KIND>
__device__ __forceinline__ void know(const SeqProb& P, ShareWalk<KIND>& w, DeviceErr* err) {
  if (w.known == w.seq) return;
  if (w.seq >= 0) w.s = seq_info(P, w.seq, err);
  w.it = items_of<KIND>(P, w.seq < 0, w.s);
  w.known = w.seq;
}
template <int KIND>
__device__ __forceinline__ void start_walk(const SeqProb& P, const SharePlan& plan, ShareWalk<KIND>& w) {
  const long long share = share_of(plan.total, gridDim.x);
  w.at = share * blockIdx.x;
  w.end = min(plan.total, w.at + share);
  w.seq = plan.first_seq;
  w.start = w.seq < 0 ? 0 : plan.first_start;
  w.kvh = w.u = 0;
  w.known = -2;
  w.s = SeqInfo{};
  if (w.at >= w.end) {
    w.start = w.end;
    return;
  }
  if (w.seq < 0 && P.shared == 0) w.seq = 0;
  know<KIND>(P, w, nullptr);
  if (w.it.count == 0) return;
  const long long all = w.it.all();
  w.kvh = quotient(w.at - w.start, all);
  w.start += w.kvh * all;
  int lo = 0, hi = w.it.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (w.it.before(mid) <= w.at - w.start) lo = mid; else hi = mid - 1;
  }
  w.u = lo;
  w.start += w.it.before(lo);
}
// The next part of the share; false at its end.
template <int KIND>
__device__ __forceinline__ bool next_share_part(const SeqProb& P, const SharePlan& plan, ShareWalk<KIND>& w, SharePart& p,
                                                DeviceErr* err) {
  using K = Kind<KIND>;
  while (w.start < w.end && w.seq < P.n_seqs) {
    know<KIND>(P, w, err);
    if (w.u >= w.it.count) {
      w.u = 0;
      ++w.kvh;
    }
    if (w.kvh >= P.Hkv || w.it.count == 0) {
      ++w.seq;
      w.kvh = w.u = 0;
      continue;
    }
    const long long a = w.start + K::W_ITEM;   // the item's first tile
    const int span = w.it.span(w.u), T = ceil_div(span, K::TILE);
    w.start = a + span;
    p.item = w.u++;
    auto tile_at = [&](long long x) { return ((int)max(0ll, min(x - a, (long long)T * K::TILE)) + K::TILE - 1) / K::TILE; };
    p.t0 = tile_at(w.at);
    p.t1 = tile_at(w.end);
    if (p.t0 >= p.t1) continue;
    p.lead = w.seq < 0;
    p.tokens = w.it.tokens;
    p.kvh = w.kvh;
    p.slot = 2 * blockIdx.x + (p.t0 > 0 ? 0 : 1);   // 0: began in an earlier CTA, 1: goes on in a later one
    p.out = (p.t0 > 0 || p.t1 < T) ? OUT_SLOT : (P.shared == 0 ? OUT_FINAL : (p.lead ? OUT_LEAD : OUT_OWN));
    p.parts = quotient(a + (long long)(T - 1) * K::TILE, w.end - w.at) - (int)blockIdx.x + 1;
    return true;
  }
  return false;
}

// What the join needs to know of an item that goes on behind a CTA's share
// (no shared region: rows are joined by item).
struct SplitItem {
  int parts;             // CTAs it is spread over; 0: none goes on
  int token, tokens;     // its first token and how many
  int kvh;
};

// ---------------------------------------------------------------- rows
// How many keys of the shared region a query token sees.
static __device__ __noinline__ int lead_limit(const SeqProb& P, int len, int token) {
  const SeqInfo s = seq_info(P, seq_of_token(P, token), nullptr);
  return clampi(token - s.q0 + 1 + s.L - s.Lq, 0, len);
}
// The same for a region of `len` keys; own regions: offset `off`, `token` counted in the sequence.
__device__ __forceinline__ int row_limit(const SeqProb& P, int lead, int off, int len, int token) {
  if (lead) return lead_limit(P, len, token);
  return P.causal ? clampi(token + 1 + off, 0, len) : len;
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}
// Exponent field of a 16-bit value all ones: infinity or NaN.
template <bool BF16>
__device__ __forceinline__ bool nonfinite16(uint32_t h) {
  constexpr uint32_t E = BF16 ? 0x7F80u : 0x7C00u;
  return (h & E) == E;
}
template <bool BF16>
__device__ __forceinline__ float widen16(uint32_t h) {
  if constexpr (BF16) return __uint_as_float(h << 16);
  return __half2float(__ushort_as_half((unsigned short)h));
}

__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Where the V rows of a region lie.
struct VRegion {
  int key0, row, kvh;    // first key (packed row, or position in table row `row`), key head
};
__device__ __forceinline__ const uint8_t* v_row(const SeqProb& P, const VRegion& g, int key) {
  const int k = g.key0 + key;
  if (!P.paged) return P.v + (long long)k * P.v_tok + g.kvh * P.v_head;
  const int page = P.table[(long long)g.row * P.max_pages + (k >> P.page_shift)];
  if ((uint32_t)page >= (uint32_t)P.n_pages) return nullptr;
  return P.v + page * P.v_page + (k & (P.page_size - 1)) * P.v_tok + g.kvh * P.v_head;
}

// The non-finite elements of V that were taken out of the products, for a row
// that sees them: N channels from c0 on, over keys [from, to).
template <bool BF16, int N>
__device__ __noinline__ void add_nonfinite(const SeqProb& P, VRegion g, int from, int to, int c0, float* y) {
  for (int key = from; key < to; ++key) {
    const uint8_t* vp = v_row(P, g, key);
    if (vp == nullptr) continue;
    const uint32_t* x = reinterpret_cast<const uint32_t*>(vp + 2 * c0);
    for (int e = 0; e < N / 2; ++e) {
      const uint32_t w = x[e];
      if (nonfinite16<BF16>(w)) y[2 * e] += widen16<BF16>(w & 0xffffu);
      if (nonfinite16<BF16>(w >> 16)) y[2 * e + 1] += widen16<BF16>(w >> 16);
    }
  }
}

// Whether a row's result lies in its buffer (the test build's self-check).
__device__ __forceinline__ bool row_inside(const SeqProb& P, const ShareBuf& b, int kind, int slot, int token, int head,
                                           int slot_row, int slot_rows) {
  return token >= 0 && token < P.total_q && head >= 0 && head < P.Hq && (kind != OUT_FINAL || !P.shared) &&
         (kind < OUT_LEAD || P.shared) &&
         (kind != OUT_SLOT || (slot >= 0 && slot < 2 * b.grid && slot_row >= 0 && slot_row < slot_rows));
}

// Where a row's result goes.
struct RowOut {
  uint8_t* h;     // final row in the output's type, or
  float* f;       // partial row
  float* lse;     // (may be NULL for a final row)
};
__device__ __forceinline__ RowOut row_out(const SeqProb& P, const ShareBuf& b, int kind, int slot, int token, int head,
                                          int slot_row, int slot_rows = SLOT_ROWS) {
  const long long grow = (long long)token * P.Hq + head;
  RowOut r;
  if (kind == OUT_FINAL) {
    r.h = P.o + token * P.o_tok + head * P.o_head;
    r.f = nullptr;
    r.lse = P.lse != nullptr ? P.lse + grow : nullptr;
    return r;
  }
  const long long at = kind == OUT_SLOT ? (long long)slot * slot_rows + slot_row : grow;
  r.h = nullptr;
  r.f = (kind == OUT_SLOT ? b.slot_o : kind == OUT_LEAD ? P.lead_o : P.own_o) + at * D;
  r.lse = (kind == OUT_SLOT ? b.slot_lse : kind == OUT_LEAD ? P.lead_lse : P.own_lse) + at;
  return r;
}
template <bool BF16>
__device__ __forceinline__ void store8(const RowOut& r, int c0, const float* y) {
  if (r.h != nullptr) {
    *reinterpret_cast<uint4*>(r.h + 2 * c0) =
        make_uint4(pack2<BF16>(y[0], y[1]), pack2<BF16>(y[2], y[3]), pack2<BF16>(y[4], y[5]), pack2<BF16>(y[6], y[7]));
  } else {
    reinterpret_cast<float4*>(r.f + c0)[0] = make_float4(y[0], y[1], y[2], y[3]);
    reinterpret_cast<float4*>(r.f + c0)[1] = make_float4(y[4], y[5], y[6], y[7]);
  }
}

}  // namespace ra
