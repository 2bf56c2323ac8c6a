// ra_packed.cu -- attention over packed sequences of different lengths
// (prompts), and over the pages of a cache whose leading tokens a batch
// shares (decoding), with grouped heads, on the sm_100a tensor cores.
//
// Mathematics: for query token i of a sequence with Lq query and L key tokens
//   o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = 2^(c (q_i . k_j) - m_i),
// c = scale log2(e), over j < limit_i (causal: limit_i = i + 1 + L - Lq),
// m_i any number near the row's maximum.  Partial results over disjoint key
// ranges join by their log-sum-exp.
//
// Work item: a pair of 128-row query tiles A, B of one key head.  Row r of a
// tile is token r / G, query head r % G of the group, so that the G heads
// that share a key head share its K and V tiles, short prompts fill rows with
// heads, and a single token's G rows need one pass over its keys.
//
// Every CTA is persistent (one per SM) and walks a list of segments: (item,
// range of 128-key tiles).  Two ways to deal them out:
//   whole items  one item per CTA in rounds, there and back; the last (longest)
//                query tiles of each sequence come first.  Rows are final.
//   split        all key tiles of all items, laid end to end, are cut into
//                equal shares, one per CTA, whatever the lengths are; an item
//                that crosses a border leaves partial rows (fp32) that
//                combine_kernel joins.  For few rows over many keys, and
//                wherever there is a shared region.
//
// 384 threads, the pipeline of the FP16 fallback kernel:
//   warps 0-3 / 4-7   softmax of tile A / B; thread t = row t = TMEM lane t
//   warp 8            segment list, Q and K copies
//   warp 11           V copies
//   warps 9, 10       MMA issuers of tile A / B (warp 9 owns TMEM)
// Copies are TMA tiles straight from the caller's tensors (any token and head
// strides), 64 channels wide with the 128-byte swizzle; a 128-key tile of a
// cache is one box per page and half.  V keeps its [key][channel] order and
// is the P.V product's N-major B operand, so nothing is transposed.
// TMEM: S_A | S_B | O_A | O_B, 128 fp32 columns each; P overwrites the upper
// half of S as 16-bit pairs and is the A operand of the P.V product.
//
// Precision: S, the row statistics, O and partial rows are fp32.  P is
// rounded to the type of V (the tensor core wants both operands alike):
// half a step of the type per weight, the size of the output's own rounding.
// The row maximum is only followed when it rises by more than 8 (powers of
// two), so O is rarely rescaled; fp16 weights carry a factor 2^7 (at most
// 2^15), which keeps weights down to 2^-31 of the largest from vanishing.
//
// Keys past a row's limit: their scores are replaced by -inf whatever they
// are.  Their V rows still meet a zero weight, and 0 x NaN is NaN, so in
// every tile that some row sees in part the softmax warps clear V rows past
// the region's end (the next sequence's rows, unwritten slots of a page) and
// replace non-finite elements by zero, remembering the tile; the epilogue
// then adds such elements back to the rows that do see them.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "ra_serve.h"

namespace ra {
namespace {

constexpr int NUM_THREADS = 384;
constexpr int STAGES = 2;
constexpr int LAUNCH_REGS = 168, SOFTMAX_REGS = 208, ISSUE_REGS = 88;
static_assert(256 * SOFTMAX_REGS + 128 * ISSUE_REGS <= NUM_THREADS * LAUNCH_REGS, "register split");
constexpr float LN2 = 0.6931471805599453f;
constexpr float RAISE = 8.0f;    // follow the row maximum when it rises by more than this (log2)
constexpr int NO_TILE = 0x7fffffff;

struct Smem {
  static constexpr uint32_t QA = 0, QB = 32768;   // 32 KB each: two 16 KB swizzled halves of 64 channels
  static constexpr uint32_t K = 65536;            // STAGES x 32 KB
  static constexpr uint32_t V = 131072;           // STAGES x 32 KB
  static constexpr uint32_t MISC = 196608;
  static constexpr uint32_t BYTES = MISC + 2048;
};

enum : int {
  B_KFULL = 0, B_KEMPTY = 2, B_VFULL = 4, B_VEMPTY = 6, B_QFULL = 8, B_QEMPTY = 9, B_SFULL = 10, B_PFULL = 12,
  B_ODONE = 16, B_DRAIN = 18, B_TURN = 20, B_SEGFULL = 22, B_SEGEMPTY = 26, NBAR = 30
};
constexpr int SEGS = 4;           // segments in flight
constexpr int SEG_READERS = 11;   // 8 softmax warps, 2 issuers, the V copier

enum : int { OUT_FINAL = 0, OUT_SLOT = 1, OUT_LEAD = 2, OUT_OWN = 3 };

// A segment, as the list warp publishes it.
struct Seg {
  int stop;
  int lead;          // 1: the shared region
  int row;           // paged: table row the keys come from
  int q0;            // first token of the sequence (lead: 0)
  int tok, ntok;     // the item's tokens: [q0 + tok, q0 + tok + ntok)
  int kvh;
  int tile0;         // first key tile
  int n[2];          // tiles that query tile A / B needs
  int nload;         // tiles that are copied: max(n[0], n[1])
  int ring;          // copies before this segment
  int qidx;          // Q copies before this segment
  int key0;          // packed: first key row of the sequence; paged: first key of the region
  int len;           // keys in the region
  int off;           // own region: limit of token t = clamp(t + 1 + off, 0, len) where causal
  int out, slot;
};

struct Misc {
  uint64_t bar[NBAR];
  uint32_t tmem;
  int abort_flag;
  int nf_tile[SEGS];         // per segment: first tile with repaired V elements
  Seg seg[SEGS];
  long long scan[13];
  long long best[13];
  long long total, first_start;
  int first_seq;
  int lead_row, lead_len;
};
static_assert(sizeof(Misc) <= 2048, "misc");

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
      if (L >= 0 && (L + P.page_size - 1) >> P.page_shift <= P.max_pages) {
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
__device__ __forceinline__ int clampi(int x, int lo, int hi) { return min(max(x, lo), hi); }

// Key tiles of a sequence's own region per item, at least one so that rows
// without keys are written too.
__device__ __forceinline__ int own_tiles(const SeqInfo& s) { return max(1, (s.len + KEYS - 1) / KEYS); }
__device__ __forceinline__ int pairs_of(const SeqProb& P, const SeqInfo& s) { return ceil_div(s.Lq, 2 * P.TQ); }

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

__device__ __forceinline__ long long lead_tiles(const SeqProb& P) { return (P.shared + KEYS - 1) / KEYS; }
__device__ __forceinline__ long long lead_total(const SeqProb& P) {
  return lead_tiles(P) * P.Hkv * ceil_div(P.total_q, 2 * P.TQ);
}

// ---------------------------------------------------------------- PTX
__device__ __forceinline__ void tma_load4(void* dst, const CUtensorMap* map, int c0, int c1, int c2, int c3,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void umma_f16_tmem_a(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                                uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// K-major operand tile (two 64-channel halves of 128-byte rows) and the
// descriptor's step to K step kk (16 channels), both in units of 16 bytes.
__device__ __forceinline__ uint64_t kmajor_desc(uint32_t base) { return sw128_desc(base); }
__host__ __device__ constexpr uint64_t kmajor_step(int kk) { return (kk >> 2) * (16384 >> 4) + (kk & 3) * (32 >> 4); }
// N-major operand tile: rows (keys) of 128 bytes hold 64 channels, 8-key
// groups 1024 bytes apart (stride offset), the two 64-channel halves 16384
// bytes apart (leading offset); a K step is 16 keys, 2048 bytes.
__device__ __forceinline__ uint64_t nmajor_desc(uint32_t base) {
  return (uint64_t)((base >> 4) & 0x3FFFu) | ((uint64_t)(16384u >> 4) << 16) | ((uint64_t)(1024u >> 4) << 32) |
         ((uint64_t)1u << 46) | ((uint64_t)2u << 61);
}
// One lane of a converged warp, the same one each time.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
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

// ---------------------------------------------------------------- segment list
// The list warp's walk; every lane holds the same values.
struct Walk {
  long long at, end;     // split: tiles of this CTA's share still to come; whole: first item of the next round
  int seq;               // split: sequence that `at` lies in; whole: round
  long long start;       // split: its first tile
};

__device__ __forceinline__ void fill_counts(const SeqProb& P, Seg& g, int tile0, int ntile) {
  g.tile0 = tile0;
#pragma unroll
  for (int X = 0; X < 2; ++X) {
    const int nt = clampi(g.ntok - X * P.TQ, 0, P.TQ);
    int n = 0;
    if (nt > 0) {
      const int last = g.tok + X * P.TQ + nt - 1;
      const int lim = (g.lead || !P.causal) ? g.len : clampi(last + 1 + g.off, 0, g.len);
      n = clampi((lim + KEYS - 1) / KEYS - tile0, 0, ntile);
    }
    g.n[X] = n;
  }
  g.nload = max(g.n[0], g.n[1]);
}

// The next segment of this CTA, or g.stop.
__device__ __forceinline__ void next_segment(const SeqProb& P, const Misc* mi, Walk& w, Seg& g, DeviceErr* err) {
  g.stop = 0;
  if (!P.split) {
    const int per = 2 * P.TQ;
    while (w.at < P.items) {
      // rounds of one item per CTA, every other one backwards: items get
      // shorter along the list, and this evens out what each CTA gets
      const long long item = w.at + (w.seq & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
      w.at += gridDim.x;
      ++w.seq;
      if (item >= P.items) continue;
      const long long pr = P.items / P.Hkv - 1 - item / P.Hkv;
      g.kvh = (int)(item % P.Hkv);
      // sequence i's pairs lie at cu_q[i] / per + i and on (never more than
      // the gap to the next sequence's first)
      int lo = 0, hi = P.n_seqs - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (P.cu_q[mid] / per + mid <= pr) lo = mid; else hi = mid - 1;
      }
      const SeqInfo s = seq_info(P, lo, err);
      const long long u = pr - (s.q0 / per + lo);
      if (u < 0 || u >= pairs_of(P, s)) continue;
      g.lead = 0;
      g.row = s.row;
      g.q0 = s.q0;
      g.tok = (int)u * per;
      g.ntok = min(per, s.Lq - g.tok);
      g.key0 = P.paged ? P.shared : s.k0;
      g.len = s.len;
      g.off = s.off;
      g.out = OUT_FINAL;
      g.slot = 0;
      fill_counts(P, g, 0, 1 << 30);
      return;
    }
    g.stop = 1;
    return;
  }
  const long long lead_all = lead_total(P);
  while (w.at < w.end) {
    long long a;         // the item's first tile
    int T;
    if (w.at < lead_all) {
      T = (int)lead_tiles(P);
      const long long item = w.at / T;
      const int pairs = ceil_div(P.total_q, 2 * P.TQ);
      a = item * T;
      g.lead = 1;
      g.kvh = (int)(item / pairs);
      g.row = mi->lead_row;
      g.q0 = 0;
      g.tok = (int)(item % pairs) * 2 * P.TQ;
      g.ntok = min(2 * P.TQ, P.total_q - g.tok);
      g.key0 = 0;
      g.len = min(P.shared, mi->lead_len);
      g.off = 0;
    } else {
      const SeqInfo s = seq_info(P, w.seq, err);
      const int pairs = pairs_of(P, s);
      T = own_tiles(s);
      const long long total = (long long)T * pairs * P.Hkv;
      if (w.at >= w.start + total) {
        w.start += total;
        if (++w.seq >= P.n_seqs) break;
        continue;
      }
      const long long item = (w.at - w.start) / T;
      a = w.start + item * T;
      g.lead = 0;
      g.kvh = (int)(item / pairs);
      g.row = s.row;
      g.q0 = s.q0;
      g.tok = (int)(item % pairs) * 2 * P.TQ;
      g.ntok = min(2 * P.TQ, s.Lq - g.tok);
      g.key0 = P.paged ? P.shared : s.k0;
      g.len = s.len;
      g.off = s.off;
    }
    const int t0 = (int)(w.at - a);
    const int t1 = (int)min((long long)T, w.end - a);
    w.at = a + t1;
    g.slot = 2 * blockIdx.x + (t0 > 0 ? 0 : 1);   // 0: began in an earlier CTA, 1: goes on in a later one
    g.out = (t0 > 0 || t1 < T) ? OUT_SLOT : (P.shared == 0 ? OUT_FINAL : (g.lead ? OUT_LEAD : OUT_OWN));
    fill_counts(P, g, t0, t1 - t0);
    return;
  }
  g.stop = 1;
}

// Lays all items' tiles end to end: the totals, and the sequence in which
// this CTA's share begins.  All threads.
__device__ void plan_split(const SeqProb& P, Misc* mi, DeviceErr* err, long long& share, long long& total) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = ceil_div(P.n_seqs, NUM_THREADS);
  const int i0 = min(P.n_seqs, tid * per), i1 = min(P.n_seqs, i0 + per);
  long long sum = 0, best = -1;
  for (int i = i0; i < i1; ++i) {
    const SeqInfo s = seq_info(P, i, err);
    sum += (long long)own_tiles(s) * pairs_of(P, s) * P.Hkv;
    // the longest sequence, the first of them, gives the shared pages
    best = max(best, ((long long)s.L << 32) | (uint32_t)(0x7fffffff - i));
  }
  long long incl = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += x;
    best = max(best, __shfl_xor_sync(0xffffffffu, best, d));
  }
  if (lane == 31) mi->scan[warp] = incl;
  if (lane == 0) mi->best[warp] = best;
  __syncthreads();
  if (tid == 0) {
    long long run = 0;
    for (int w = 0; w < NUM_THREADS / 32; ++w) {
      const long long x = mi->scan[w];
      mi->scan[w] = run;
      run += x;
      best = max(best, mi->best[w]);
    }
    mi->total = run;
    const int i = 0x7fffffff - (int)(uint32_t)(best & 0xffffffffll);
    const SeqInfo s = seq_info(P, i, err);
    mi->lead_row = s.row;
    mi->lead_len = s.L;
    mi->first_seq = 0;
    mi->first_start = lead_total(P);
  }
  __syncthreads();
  const long long lead = lead_total(P);
  total = lead + mi->total;
  share = (total + gridDim.x - 1) / gridDim.x;
  const long long mine = share * blockIdx.x;
  long long at = lead + mi->scan[warp] + incl - sum;
  if (blockIdx.x == 0 || (mine >= at && mine < at + sum)) {
    for (int i = i0; i < i1; ++i) {
      const SeqInfo s = seq_info(P, i, nullptr);
      const long long n = (long long)own_tiles(s) * pairs_of(P, s) * P.Hkv;
      if (blockIdx.x == 0) P.starts[i] = at;
      if (mine >= at && mine < at + n) {
        mi->first_seq = i;
        mi->first_start = at;
      }
      at += n;
    }
    if (blockIdx.x == 0 && i1 == P.n_seqs && i0 < i1) P.starts[P.n_seqs] = at;
  }
  __syncthreads();
}

// Address of V element (key, channel 0) of a segment's region.
__device__ __forceinline__ const uint8_t* v_row(const SeqProb& P, const Seg& g, int key) {
  if (!P.paged) return P.v + (long long)(g.key0 + key) * P.v_tok + g.kvh * P.v_head;
  const int k = g.key0 + key;
  const int page = P.table[(long long)g.row * P.max_pages + (k >> P.page_shift)];
  if ((uint32_t)page >= (uint32_t)P.n_pages) return nullptr;
  return P.v + page * P.v_page + (k & (P.page_size - 1)) * P.v_tok + g.kvh * P.v_head;
}

template <bool BF16>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    seq_attn_kernel(const __grid_constant__ SeqProb P, const __grid_constant__ CUtensorMap mq,
                    const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                    WsHeader* __restrict__ hdr, uint64_t limit_ns) {
  constexpr float BIAS = BF16 ? 0.0f : 7.0f;
  constexpr uint32_t FMT = BF16 ? 1 : 0;
  constexpr uint32_t IDESC_S = make_idesc(1, FMT, FMT, 128, 128);
  constexpr uint32_t IDESC_PV = make_idesc(1, FMT, FMT, 128, 128) | (1u << 16);   // B is N-major
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = align1024(smem_raw);
  Misc* mi = reinterpret_cast<Misc*>(sm + Smem::MISC);
  uint64_t* bar = mi->bar;
  volatile int* abort_flag = &mi->abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  DeviceErr* err = &hdr->err;

  if (tid == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&bar[B_KFULL + i], 1);
      mbar_init(&bar[B_KEMPTY + i], 2);
      mbar_init(&bar[B_VFULL + i], 1);
      mbar_init(&bar[B_VEMPTY + i], 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar[B_SFULL + i], 1);
      mbar_init(&bar[B_PFULL + i], 4);       // first half of P, tile A / B
      mbar_init(&bar[B_PFULL + 2 + i], 4);   // second half
      mbar_init(&bar[B_ODONE + i], 1);
      mbar_init(&bar[B_DRAIN + i], 1);
      mbar_init(&bar[B_TURN + i], 1);
    }
    for (int i = 0; i < SEGS; ++i) {
      mbar_init(&bar[B_SEGFULL + i], 1);
      mbar_init(&bar[B_SEGEMPTY + i], SEG_READERS);
    }
    mbar_init(&bar[B_QFULL], 1);
    mbar_init(&bar[B_QEMPTY], 2);
    mi->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(&mi->tmem, 512);
    tmem_relinquish();
  }
  long long share = 0, total = 0;
  if (P.split) plan_split(P, mi, err, share, total);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = mi->tmem;
  if (warp < 8) {
    regs_inc<SOFTMAX_REGS>();
  } else {
    regs_dec<ISSUE_REGS>();
  }
  auto wait = [&](int b, uint32_t parity, uint32_t site) {
    return mbar_wait_abortable(&bar[b], parity, abort_flag, limit_ns, err, site);
  };
  auto wait_all = [&](int b, uint32_t parity, uint32_t site) {
    return __all_sync(0xffffffffu, wait(b, parity, site)) != 0;
  };
  // Segment k, once it is published; a reader warp frees its place when it no
  // longer reads it.
  auto segment = [&](int k, uint32_t site) -> const Seg* {
    return wait_all(B_SEGFULL + k % SEGS, (k / SEGS) & 1, site) ? &mi->seg[k % SEGS] : nullptr;
  };
  auto free_segment = [&](int k) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar[B_SEGEMPTY + k % SEGS]);
  };

  if (warp < 8) {
    // ------------------------------------------------------------ softmax
    const int X = warp >> 2, wq = warp & 3, r = tid & 127;
    const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
    const uint32_t tS = tbase + X * 128 + lane_off, tO = tbase + 256 + X * 128 + lane_off;
    const float cs = P.cs;
    const int rtok = r / P.G, rhead = r % P.G;
    uint32_t s_phase = 0, o_phase = 0;
    for (int k = 0;; ++k) {
      const Seg* seg = segment(k, 0x4101);
      if (seg == nullptr || seg->stop) break;
      const Seg& g = *seg;
      const int n = X ? g.n[1] : g.n[0];
      const int tt = g.tok + X * P.TQ + rtok;              // token within the sequence (lead: within all)
      const bool valid = rtok < P.TQ && X * P.TQ + rtok < g.ntok;
      if (X * P.TQ >= g.ntok) {                            // no tile B in this item
        free_segment(k);
        continue;
      }
      // this row's limit, and the smallest of the tile's (the same in its four warps)
      const int t0 = g.tok + X * P.TQ, t1 = min(t0 + P.TQ, g.tok + g.ntok);
      int lim, gmin;
      if (g.lead) {
        auto limit_of = [&](int t) {
          const SeqInfo s = seq_info(P, seq_of_token(P, t), nullptr);
          return clampi(t - s.q0 + 1 + s.L - s.Lq, 0, g.len);
        };
        lim = valid ? limit_of(tt) : 0;
        gmin = g.len;
        for (int t = t0 + lane; t < t1; t += 32) gmin = min(gmin, limit_of(t));
        gmin = __reduce_min_sync(0xffffffffu, gmin);
      } else {
        lim = P.causal ? clampi(tt + 1 + g.off, 0, g.len) : g.len;
        gmin = P.causal ? clampi(t0 + 1 + g.off, 0, g.len) : g.len;
      }
      const bool active = __any_sync(0xffffffffu, valid);
      float m = -INFINITY, l = 0.0f;
      bool ok = true;
      for (int t = 0; t < n; ++t) {
        const int key = (g.tile0 + t) * KEYS;
        // S(t) has landed -- and with it P.V(t-1)
        if (!(ok = wait_all(B_SFULL + X, s_phase & 1, 0x4102))) break;
        ++s_phase;
        if (gmin < key + KEYS) {
          // a tile that some row sees in part: this warp's 32 V rows
          const int ring = g.ring + t;
          if (!(ok = wait_all(B_VFULL + ring % STAGES, (ring / STAGES) & 1, 0x4103))) break;
          uint8_t* vt = sm + Smem::V + (ring % STAGES) * 32768;
          const int vr = 32 * wq + lane;
          uint4* h0 = reinterpret_cast<uint4*>(vt + vr * 128);
          uint4* h1 = reinterpret_cast<uint4*>(vt + 16384 + vr * 128);
          if (key + vr >= g.len) {
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              h0[(c + lane) & 7] = make_uint4(0, 0, 0, 0);
              h1[(c + lane) & 7] = make_uint4(0, 0, 0, 0);
            }
          } else {
            for (int c = 0; c < 16; ++c) {
              uint4* at = (c < 8 ? h0 : h1) + ((c + lane) & 7);
              uint4 w = *at;
              uint32_t* x = reinterpret_cast<uint32_t*>(&w);
              bool bad = false;
#pragma unroll
              for (int e = 0; e < 4; ++e) bad |= nonfinite16<BF16>(x[e] & 0xffffu) || nonfinite16<BF16>(x[e] >> 16);
              if (bad) {
                atomicMin(&mi->nf_tile[k % SEGS], g.tile0 + t);
                __threadfence_block();
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  if (nonfinite16<BF16>(x[e] & 0xffffu)) x[e] &= 0xffff0000u;
                  if (nonfinite16<BF16>(x[e] >> 16)) x[e] &= 0xffffu;
                }
                *at = w;
              }
            }
          }
          fence_async_smem();
          __syncwarp();
        }
        if (active) {
          tc_fence_after();
          uint32_t s[128];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(tS + 32 * c, s + 32 * c);
          tmem_wait_ld();
          const int nvalid = lim - key;
          if (__any_sync(0xffffffffu, nvalid < KEYS)) {
#pragma unroll
            for (int e = 0; e < 128; ++e)
              if (e >= nvalid) s[e] = 0xFF800000u;   // -inf: out of the max and the sum
          }
          // a NaN score makes the maximum, and so the row, NaN
          float mh[8];
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            mh[c] = max3_nan(__uint_as_float(s[16 * c]), __uint_as_float(s[16 * c + 1]), __uint_as_float(s[16 * c + 2]));
#pragma unroll
            for (int e = 3; e < 15; e += 2)
              mh[c] = max3_nan(mh[c], __uint_as_float(s[16 * c + e]), __uint_as_float(s[16 * c + e + 1]));
          }
#pragma unroll
          for (int c = 0; c < 8; c += 2)
            mh[c] = max3_nan(max3_nan(mh[c], mh[c + 1], __uint_as_float(s[16 * c + 15])), __uint_as_float(s[16 * c + 31]), mh[c]);
          const float mx = max3_nan(max3_nan(mh[0], mh[2], mh[4]), mh[6], mh[6]) * cs;
          const bool moved = !(mx <= m + RAISE);       // from -inf: as soon as a key is seen
          const float m_new = moved ? (mx == INFINITY ? NAN : mx) : m;   // an infinite score: inf - inf
          const float alpha = moved ? ex2(m - m_new) : 1.0f;
          m = m_new;
          const float add = BIAS - (m == -INFINITY ? 0.0f : m);
          if (t > 0 && __any_sync(0xffffffffu, moved)) {
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              uint32_t acc[32];
              tmem_ld32(tO + 32 * c, acc);
              tmem_wait_ld();
              if (moved) {
#pragma unroll
                for (int e = 0; e < 32; ++e) acc[e] = __float_as_uint(__uint_as_float(acc[e]) * alpha);
              }
              tmem_st32(tO + 32 * c, acc);
            }
          }
          float l0 = 0.0f, l1 = 0.0f;
          // P in two halves: the first one's product starts under the second one's exponentials
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t ph[32];
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              const int e = 64 * half + 2 * c;
              float x0, x1;
              fma2(x0, x1, __uint_as_float(s[e]), __uint_as_float(s[e + 1]), cs, cs, add, add);
              const float p0 = ex2(x0), p1 = ex2(x1);
              add2(l0, l1, l0, l1, p0, p1);
              ph[c] = pack2<BF16>(p0, p1);
            }
            tmem_st32(tS + 64 + 32 * half, ph);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[B_PFULL + 2 * half + X]);
          }
          l = fmaf(l, alpha, l0 + l1);
        } else {
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&bar[B_PFULL + X]);
            mbar_arrive(&bar[B_PFULL + 2 + X]);
          }
        }
      }
      if (!ok) break;
      if (n > 0) {
        if (!wait_all(B_ODONE + X, o_phase & 1, 0x4104)) break;
        ++o_phase;
      }
      if (!active) {
        free_segment(k);
        continue;
      }
      // epilogue: rows of this segment, final or partial
      tc_fence_after();
      const float inv = l != 0.0f ? 1.0f / l : 0.0f;
      const float lse2 = l != 0.0f ? m - BIAS + log2f(l) : -INFINITY;
      const int token = g.q0 + tt, head = g.kvh * P.G + rhead;
      const bool store = valid && in_bounds(token >= 0 && token < P.total_q && head < P.Hq, err, 0x4105);
      const long long grow = (long long)token * P.Hq + head;
      const int nf = *reinterpret_cast<volatile int*>(&mi->nf_tile[k % SEGS]);
      float* frow = nullptr;
      uint8_t* hrow = nullptr;
      if (g.out == OUT_FINAL) {
        hrow = P.o + token * P.o_tok + head * P.o_head;
        if (store && P.lse != nullptr) P.lse[grow] = lse2 * LN2;
      } else {
        const long long at = g.out == OUT_SLOT ? (long long)g.slot * SLOT_ROWS + X * 128 + r : grow;
        frow = (g.out == OUT_SLOT ? P.slot_o : g.out == OUT_LEAD ? P.lead_o : P.own_o) + at * D;
        float* lrow = (g.out == OUT_SLOT ? P.slot_lse : g.out == OUT_LEAD ? P.lead_lse : P.own_lse) + at;
        if (store) *lrow = lse2;
      }
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        float y[32];
        if (n > 0) {
          uint32_t acc[32];
          tmem_ld32(tO + 32 * c, acc);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) y[e] = l != 0.0f ? __uint_as_float(acc[e]) * inv : 0.0f;
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) y[e] = 0.0f;
        }
        if (nf != NO_TILE && store) {
          // non-finite elements of V that were taken out of the product, for
          // the rows that see them
          const int last = min(lim, (g.tile0 + n) * KEYS);
          for (int key = nf * KEYS; key < last; ++key) {
            const uint8_t* vp = v_row(P, g, key);
            if (vp == nullptr) continue;
            const uint32_t* x = reinterpret_cast<const uint32_t*>(vp + 64 * c);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const uint32_t w = x[e];
              if (nonfinite16<BF16>(w & 0xffffu)) y[2 * e] += widen16<BF16>(w & 0xffffu);
              if (nonfinite16<BF16>(w >> 16)) y[2 * e + 1] += widen16<BF16>(w >> 16);
            }
          }
        }
        if (store) {
          if (hrow != nullptr) {
            uint4* dst = reinterpret_cast<uint4*>(hrow + 64 * c);
#pragma unroll
            for (int q = 0; q < 4; ++q)
              dst[q] = make_uint4(pack2<BF16>(y[8 * q], y[8 * q + 1]), pack2<BF16>(y[8 * q + 2], y[8 * q + 3]),
                                  pack2<BF16>(y[8 * q + 4], y[8 * q + 5]), pack2<BF16>(y[8 * q + 6], y[8 * q + 7]));
          } else {
            float4* dst = reinterpret_cast<float4*>(frow + 32 * c);
#pragma unroll
            for (int q = 0; q < 8; ++q) dst[q] = make_float4(y[4 * q], y[4 * q + 1], y[4 * q + 2], y[4 * q + 3]);
          }
        }
      }
      tc_fence_before();   // O has been read: the next segment's first P.V follows this row's next P
      free_segment(k);
    }
  } else if (warp == 8 || warp == 11) {
    // ------------------------------------------------------------ copies
    const bool isK = warp == 8;
    const int FULL = isK ? B_KFULL : B_VFULL, EMPTY = isK ? B_KEMPTY : B_VEMPTY;
    const uint32_t base = isK ? Smem::K : Smem::V;
    const CUtensorMap* map = isK ? &mk : &mv;
    if (lane == 0) {
      asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
      if (isK) asm volatile("prefetch.tensormap [%0];" ::"l"(&mq) : "memory");
    }
    Walk w;
    if (P.split) {
      w.at = share * blockIdx.x;
      w.end = min(total, w.at + share);
      w.seq = mi->first_seq;
      w.start = mi->first_start;
    } else {
      w.at = w.end = w.start = 0;
      w.seq = 0;
    }
    int ring = 0, qidx = 0;
    bool ok = true;
    Seg g;
    for (int k = 0; ok; ++k) {
      if (isK) {
        next_segment(P, mi, w, g, err);
        g.ring = ring;
        g.qidx = qidx;
        if (k >= SEGS && !(ok = wait_all(B_SEGEMPTY + k % SEGS, (k / SEGS - 1) & 1, 0x4201))) break;
        if (lane == 0) {
          mi->seg[k % SEGS] = g;
          mi->nf_tile[k % SEGS] = NO_TILE;
          __threadfence_block();
          mbar_arrive(&bar[B_SEGFULL + k % SEGS]);
        }
        __syncwarp();
        if (g.stop) break;
        if (g.nload > 0) {
          if (qidx > 0 && !(ok = wait_all(B_QEMPTY, (qidx - 1) & 1, 0x4202))) break;
          if (lane == 0) {
            const int nq = g.n[1] > 0 ? 2 : 1;
            mbar_expect_tx(&bar[B_QFULL], nq * 2u * 128u * P.G * P.TQ);
            for (int X = 0; X < nq; ++X)
              for (int h = 0; h < 2; ++h)
                tma_load4(sm + (X ? Smem::QB : Smem::QA) + h * 16384, &mq, 64 * h, 0, g.kvh,
                          g.q0 + g.tok + X * P.TQ, &bar[B_QFULL]);
          }
          __syncwarp();
          ++qidx;
        }
      } else {
        const Seg* seg = segment(k, 0x4203);
        if (!(ok = seg != nullptr)) break;
        g = *seg;
        free_segment(k);
        if (g.stop) break;
      }
      for (int t = 0; t < g.nload; ++t, ++ring) {
        const int st = ring % STAGES;
        const int key = (g.tile0 + t) * KEYS;
        int page = 0;
        bool box = false;
        if (P.paged) {
          // lane b copies the page that holds the tile's keys b * page_size and on
          const int first = key + (lane << P.page_shift);
          box = lane < (KEYS >> P.page_shift) && first < g.len;
          if (box) {
            page = P.table[(long long)g.row * P.max_pages + ((g.key0 + first) >> P.page_shift)];
            if ((uint32_t)page >= (uint32_t)P.n_pages) {   // not a page: read as zeros
              report(err, DEVERR_BOUNDS, 0x4204);
              page = P.n_pages;
            }
          }
        }
        if (ring >= STAGES && !(ok = wait_all(EMPTY + st, ((ring / STAGES) - 1) & 1, 0x4205))) break;
        uint8_t* dst = sm + base + st * 32768;
        if (P.paged) {
          const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, box));
          if (lane == 0) mbar_expect_tx(&bar[FULL + st], boxes * 256u * P.page_size);
          __syncwarp();
          if (box) {
            uint8_t* d = dst + ((lane << P.page_shift) * 128);
            tma_load4(d, map, 0, 0, g.kvh, page, &bar[FULL + st]);
            tma_load4(d + 16384, map, 64, 0, g.kvh, page, &bar[FULL + st]);
          }
          __syncwarp();
        } else if (lane == 0) {
          mbar_expect_tx(&bar[FULL + st], 32768u);
          tma_load4(dst, map, 0, 0, g.kvh, g.key0 + key, &bar[FULL + st]);
          tma_load4(dst + 16384, map, 64, 0, g.kvh, g.key0 + key, &bar[FULL + st]);
        }
      }
    }
    // every copy lands before the CTA exits, also after another role gave up
    if (isK && qidx > 0) mbar_wait(&bar[B_QFULL], (qidx - 1) & 1, limit_ns, err, 0x4206);
    for (int t = ring > STAGES ? ring - STAGES : 0; t < ring; ++t)
      mbar_wait(&bar[FULL + t % STAGES], (t / STAGES) & 1, limit_ns, err, 0x4207);
  } else {
    // ------------------------------------------------------------ MMA issuers
    // One warp per query tile.  They take turns, tile A's P.V(t) and S(t+1),
    // then tile B's: so the tiles stay half a period apart and one tile's
    // softmax runs under the other's products.  (Without turns the two fall
    // into step, both in the exponentials, sharing their pipe, then both
    // waiting; one warp for both adds its own waits to the critical path.)
    // The warp stays converged and its addresses uniform (one elected lane
    // issues): descriptors live in uniform registers and step by additions,
    // where a lane of its own took ~100 cycles per MMA to move them there.
    const int X = __shfl_sync(0xffffffffu, warp - 9, 0);
    const uint64_t qd = kmajor_desc(smem_u32(sm + Smem::QA)) + X * (32768 >> 4);
    const uint64_t kd = kmajor_desc(smem_u32(sm + Smem::K)), vd = nmajor_desc(smem_u32(sm + Smem::V));
    const uint32_t tS = __shfl_sync(0xffffffffu, tbase, 0) + X * 128, tO = tS + 256;
    uint32_t p_phase = 0;
    int turn = 0;                  // groups of this tile so far
    auto spin_all = [&](int b, uint32_t parity, uint32_t site) {
      // polls without suspending at first, then as every other wait
#pragma unroll 1
      for (int i = 0; i < 64; ++i)
        if (__all_sync(0xffffffffu, mbar_test_wait(&bar[b], parity))) return true;
      return wait_all(b, parity, site);
    };
    auto issue_S = [&](int ring) {   // S = Q K^T
      const uint64_t kt = kd + (ring % STAGES) * (32768 >> 4);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          umma_f16(tS, qd + kmajor_step(kk), kt + kmajor_step(kk), IDESC_S, kk > 0);
        umma_commit(&bar[B_SFULL + X]);
      }
      __syncwarp();
    };
    bool ok = true;
    for (int k = 0; ok; ++k) {
      const Seg* seg = segment(k, 0x4301);
      if (!(ok = seg != nullptr)) break;
      const Seg& g = *seg;
      const int nload = __shfl_sync(0xffffffffu, g.nload, 0), ring0 = __shfl_sync(0xffffffffu, g.ring, 0);
      const int n = __shfl_sync(0xffffffffu, X ? g.n[1] : g.n[0], 0);
      const int q_phase = __shfl_sync(0xffffffffu, g.qidx & 1, 0), stop = __shfl_sync(0xffffffffu, g.stop, 0);
      free_segment(k);
      if (stop) break;
      if (nload == 0) continue;
      auto k_full = [&](int t) {
        return wait_all(B_KFULL + (ring0 + t) % STAGES, ((ring0 + t) / STAGES) & 1, 0x4302);
      };
      auto k_done = [&](int t, bool mma) {   // this tile's S has read K(t), or never will
        if (elect_one()) {
          if (mma) umma_commit(&bar[B_KEMPTY + (ring0 + t) % STAGES]);
          else mbar_arrive(&bar[B_KEMPTY + (ring0 + t) % STAGES]);
          if (t == nload - 1) {
            if (mma) umma_commit(&bar[B_QEMPTY]);
            else mbar_arrive(&bar[B_QEMPTY]);
          }
        }
        __syncwarp();
      };
      if (!(ok = wait_all(B_QFULL, q_phase, 0x4304) && k_full(0))) break;
      tc_fence_after();
      if (n > 0) issue_S(ring0);
      k_done(0, n > 0);
      for (int t = 0; t < nload; ++t) {
        const int ring = ring0 + t;
        const uint64_t vt = vd + (ring % STAGES) * (32768 >> 4);
        if (!(ok = wait_all(B_VFULL + ring % STAGES, (ring / STAGES) & 1, 0x4303))) break;
        if (t + 1 < nload && !(ok = k_full(t + 1))) break;
        // A goes first; its first turn needs no leave
        if (X == 1 || turn > 0) {
          if (!(ok = spin_all(B_TURN + X, (X ? turn : turn - 1) & 1, 0x4306))) break;
        }
        ++turn;
        if (t < n) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {   // O += P(t) V(t), P from TMEM
            if (!ok || !(ok = spin_all(B_PFULL + 2 * half + X, p_phase, 0x4305))) continue;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int kk = 4 * half; kk < 4 * half + 4; ++kk)
                umma_f16_tmem_a(tO, tS + 64 + 8 * kk, vt + kk * (2048 >> 4), IDESC_PV, (t > 0) || (kk > 0));
            }
            __syncwarp();
          }
          if (!ok) break;
          p_phase ^= 1u;
          if (t + 1 < n) {
            issue_S(ring + 1);
          } else {
            if (elect_one()) umma_commit(&bar[B_ODONE + X]);
            __syncwarp();
          }
        }
        if (lane == 0) mbar_arrive(&bar[B_TURN + 1 - X]);
        __syncwarp();
        if (elect_one()) {
          if (t < n) umma_commit(&bar[B_VEMPTY + ring % STAGES]);
          else mbar_arrive(&bar[B_VEMPTY + ring % STAGES]);
        }
        __syncwarp();
        if (t + 1 < nload) k_done(t + 1, t + 1 < n);
      }
    }
    if (elect_one()) umma_commit(&bar[B_DRAIN + X]);   // every MMA completes before TMEM is released
    __syncwarp();
    mbar_wait(&bar[B_DRAIN + X], 0, limit_ns, err, 0x4306);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

// Joins partial rows: one warp per (token, head), four channels per lane.
//   o = sum_s 2^(lse_s - M) o_s / sum_s 2^(lse_s - M),  M = max lse_s
// over the parts the split kernel left: the shared region's and the own
// region's, each whole or in slots of consecutive CTAs.  Memory-bound: reads
// 516 bytes per part and row, writes 256.
template <bool BF16>
__global__ void __launch_bounds__(256) combine_kernel(const __grid_constant__ SeqProb P) {
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= (long long)P.total_q * P.Hq) return;
  const int token = (int)(row / P.Hq), head = (int)(row % P.Hq);
  const int kvh = head / P.G, gh = head % P.G, per = 2 * P.TQ;
  const int i = seq_of_token(P, token);
  const SeqInfo s = seq_info(P, i, nullptr);
  if (token < s.q0 || token >= s.q0 + s.Lq) return;   // behind the last sequence
  const long long total = P.starts[P.n_seqs];
  const long long share = (total + P.grid - 1) / P.grid;
  long long a[2];        // first tile of the two regions' items
  int T[2], in[2];       // tiles; the row's index within its slot
  const int r0 = P.shared > 0 ? 0 : 1;
  {
    const int pairs = ceil_div(P.total_q, per), u = token / per, tt = token % per;
    T[0] = (int)lead_tiles(P);
    a[0] = (long long)(kvh * pairs + u) * T[0];
    in[0] = (tt / P.TQ) * 128 + (tt % P.TQ) * P.G + gh;
  }
  {
    const int t = token - s.q0, u = t / per, tt = t % per;
    T[1] = own_tiles(s);
    a[1] = P.starts[i] + (long long)(kvh * pairs_of(P, s) + u) * T[1];
    in[1] = (tt / P.TQ) * 128 + (tt % P.TQ) * P.G + gh;
  }
  if (r0 == 1 && a[1] / share == (a[1] + T[1] - 1) / share) return;   // final already
  float M = -INFINITY;
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    if (g < r0) continue;
    const float* whole_l = g ? P.own_lse : P.lead_lse;
    const long long c0 = a[g] / share, c1 = (a[g] + T[g] - 1) / share;
    if (c0 == c1) {
      M = fmaxf(M, whole_l[row]);
    } else {
      for (long long c = c0; c <= c1; ++c) M = fmaxf(M, P.slot_lse[(2 * c + (c == c0)) * SLOT_ROWS + in[g]]);
    }
  }
  float sum = 0.0f;
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (M != -INFINITY) {
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      if (g < r0) continue;
      const float *whole_o = g ? P.own_o : P.lead_o, *whole_l = g ? P.own_lse : P.lead_lse;
      const long long c0 = a[g] / share, c1 = (a[g] + T[g] - 1) / share;
      for (long long c = c0; c <= c1; ++c) {
        const long long at = c0 == c1 ? row : (2 * c + (c == c0)) * SLOT_ROWS + in[g];
        const float l = c0 == c1 ? whole_l[at] : P.slot_lse[at];
        if (l == -INFINITY) continue;                  // saw no key
        const float w = exp2f(l - M);
        const float4 x = reinterpret_cast<const float4*>((c0 == c1 ? whole_o : P.slot_o) + at * D)[lane];
        sum += w;
        acc.x = fmaf(w, x.x, acc.x);
        acc.y = fmaf(w, x.y, acc.y);
        acc.z = fmaf(w, x.z, acc.z);
        acc.w = fmaf(w, x.w, acc.w);
      }
    }
  }
  const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
  const uint2 out = make_uint2(pack2<BF16>(acc.x * inv, acc.y * inv), pack2<BF16>(acc.z * inv, acc.w * inv));
  *reinterpret_cast<uint2*>(P.o + token * P.o_tok + head * P.o_head + 8 * lane) = out;
  if (lane == 0 && P.lse != nullptr) P.lse[row] = sum != 0.0f ? (M + log2f(sum)) * LN2 : -INFINITY;
}

template <bool BF16>
cudaError_t launch(const SeqProb& p, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, void* ws,
                   cudaStream_t st) {
  const int smem = Smem::BYTES + 1024;   // > half the SM: one CTA per SM owns all 512 TMEM columns
  auto kern = seq_attn_kernel<BF16>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaFuncAttributes fa;   // the setmaxnreg split needs exactly LAUNCH_REGS at launch
  e = cudaFuncGetAttributes(&fa, kern);
  if (e != cudaSuccess) return e;
  if (fa.numRegs != LAUNCH_REGS) return cudaErrorInvalidConfiguration;
  kern<<<p.grid, NUM_THREADS, smem, st>>>(p, mq, mk, mv, static_cast<WsHeader*>(ws), wait_limit());
  e = cudaGetLastError();
  if (e != cudaSuccess || !p.split) return e;
  const long long rows = (long long)p.total_q * p.Hq;
  combine_kernel<BF16><<<(unsigned)((rows + 7) / 8), 256, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_seq_attention(const SeqProb& p, const CUtensorMap& mq, const CUtensorMap& mk,
                                 const CUtensorMap& mv, void* ws, cudaStream_t st) {
  return p.bf16 ? launch<true>(p, mq, mk, mv, ws, st) : launch<false>(p, mq, mk, mv, ws, st);
}

}  // namespace ra
