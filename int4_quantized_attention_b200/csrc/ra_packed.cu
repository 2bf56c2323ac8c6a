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
// heads, and a token's G rows need one pass over its keys.
//
// Every CTA is persistent (one per SM) and works through segments: (item,
// range of 128-key tiles).  Two ways to deal them out:
//   whole items  one at a time to the CTA that is free, those with the most key
//                tiles first.  Rows are final.
//   split        all items, laid end to end, are cut into equal shares, one per
//                CTA, whatever the lengths are; an item that crosses a border
//                leaves partial rows (fp32) that a joining kernel puts together.
//                For few items (below two per SM), and over pages.  With more,
//                whole items win, since a share's first and last rows go through
//                memory once more (packed_split in ra_serve_api.cu has the figures).
//
// 384 threads:
//   warps 0-3 / 4-7   softmax of tile A / B; thread t = row t = TMEM lane t
//   warp 8            the segment list, a few segments ahead
//   warps 9, 10       MMA issuers of tile A / B (warp 9 owns TMEM)
//   warp 11           copies
// Copies are TMA tiles straight from the caller's tensors (any token and head
// strides), 64 channels wide with the 128-byte swizzle; a 128-key tile of a
// cache is one box per page and half, one per lane.  V keeps its [key][channel]
// order and is the P.V product's N-major B operand, so nothing is transposed.
// K and V have two stages of 32 KB each.
// TMEM: S_A | S_B | O_A | O_B, 128 fp32 columns each; P overwrites the upper
// half of S as 16-bit pairs and is the A operand of the P.V product.
//
// What bounds it: from some thousand tokens on, 3340 cycles per pair of tiles,
// whose products need 2048 and whose exponentials as many (the tensor pipe is
// active 59 % of the time), at the 1.55 to 1.7 GHz that the power limit leaves
// (990 W): 980 to 1100 TFLOP/s, where a bf16 matrix product sustains 1377 at that
// limit.  Below, what a segment costs besides its tiles (a masked tile's softmax
// 3500 to 6000 cycles, the epilogue 4000).  The softmax threads spill: a 272-byte
// frame, 248 bytes of stores.
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
// every tile that some row sees in part softmax warps (tile A's, where A has
// the tile) clear V rows past the region's end (the next sequence's rows,
// unwritten slots of a page) and replace non-finite elements by zero,
// remembering the tile; the epilogue then adds such elements back to the rows
// that do see them.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "ra_seq.cuh"

namespace ra {
namespace {

constexpr int NUM_THREADS = 384;
constexpr int STAGES = 2;
constexpr int LAUNCH_REGS = 168, SOFTMAX_REGS = 216, ISSUE_REGS = 72;
static_assert(256 * SOFTMAX_REGS + 128 * ISSUE_REGS <= NUM_THREADS * LAUNCH_REGS, "register split");
constexpr int SEGS = 8;           // segments in flight
constexpr int SEG_READERS = 11;   // 8 softmax warps, 2 issuers, the copier

struct Smem {
  static constexpr uint32_t QA = 0, QB = 32768;   // 32 KB each: two 16 KB swizzled halves of 64 channels
  static constexpr uint32_t K = 65536;            // STAGES x 32 KB
  static constexpr uint32_t V = 131072;           // STAGES x 32 KB
  static constexpr uint32_t STAGE = 196608;       // 2 KB per softmax warp: rows on their way out
  static constexpr uint32_t MISC = STAGE + 16384;
  static constexpr uint32_t BYTES = MISC + 2048;
};

enum : int {
  B_KFULL = 0, B_KEMPTY = 2, B_VFULL = 4, B_VEMPTY = 6, B_QFULL = 8, B_QEMPTY = 10, B_SFULL = 12, B_PFULL = 14,
  B_ODONE = 18, B_DRAIN = 20, B_TURN = 22, B_SEGFULL = 24, B_SEGEMPTY = 32, NBAR = 40
};

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
  int qidx[2];       // copies of Q tile A / B before this segment
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
  SharePlan plan;
};
static_assert(sizeof(Misc) <= 2048, "misc");

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

// Bounded wait of a converged warp; short, since the kernel's instructions
// have to stay in the cache.  The hardware suspends the threads between tests:
// polling costs issue slots and power (32 polls first: 2 to 3 % slower from
// 8192 tokens on).  Gives up when the limit has passed or another role has.
struct Waits {
  uint64_t* bar;
  volatile int* abort_flag;
  uint64_t limit_ns;
  DeviceErr* err;
};
__device__ __noinline__ void gave_up(volatile int* abort_flag, DeviceErr* err, uint32_t site) {
  if (!*abort_flag) report(err, DEVERR_TIMEOUT, site);
  *abort_flag = 1;
}
__device__ __forceinline__ bool wait_warp(const Waits& w, int b, uint32_t parity, uint32_t site) {
  uint64_t* bar = &w.bar[b];
  if (__all_sync(0xffffffffu, mbar_test_wait(bar, parity))) return true;
  const uint64_t t0 = globaltimer_ns();
#pragma unroll 1
  while (true) {
    if (__all_sync(0xffffffffu, mbar_try_wait_sleep(bar, parity, kSleepHintNs))) return true;
    if (__any_sync(0xffffffffu, *w.abort_flag || globaltimer_ns() - t0 > w.limit_ns)) break;
  }
  gave_up(w.abort_flag, w.err, site);
  return false;
}

// ---------------------------------------------------------------- segment list
// The list warp's walk; every lane holds the same values.
__device__ __forceinline__ void fill_counts(const SeqProb& P, Seg& g, int t0, int t1) {
  g.tile0 = t0;
#pragma unroll
  for (int X = 0; X < 2; ++X) {
    const int nt = clampi(g.ntok - X * P.TQ, 0, P.TQ);
    int n = 0;
    if (nt > 0) {
      const int last = g.tok + X * P.TQ + nt - 1;
      const int lim = (g.lead || !P.causal) ? g.len : clampi(last + 1 + g.off, 0, g.len);
      n = clampi((lim + KEYS - 1) / KEYS - t0, 0, t1 - t0);
    }
    g.n[X] = n;
  }
  g.nload = max(g.n[0], g.n[1]);
}

// Whole items go out one at a time: a CTA's first is its own number, each
// later one the next that nobody has (a ticket in the workspace header, which
// the last CTA to leave sets back).  Up to LPT_SEQS sequences the list runs from
// the items with the most key tiles to those with the fewest, so that what
// remains at the end is short; beyond that from the last query tiles of the
// last sequence on.
constexpr int LPT_SEQS = 128;
struct WholeList {
  Items<KIND_MANY> it[LPT_SEQS / 32];   // this lane's sequences: lane, lane + 32, ...
  int pairs, most;                      // all pairs of query tiles; key tiles of the longest
  int round;
};
// How many of a sequence's pairs have at least T key tiles: its last ones.
__device__ __forceinline__ int pairs_from(const Items<KIND_MANY>& it, int T) {
  const int over = KEYS * (T - 1);      // keys that such a pair sees more than
  if (it.count == 0 || it.span(it.count - 1) <= over) return 0;
  if (it.step == 0 || over < it.base) return it.count;
  return it.count - min((over - it.base) / it.step, it.count - 1);
}
__device__ __forceinline__ void start_list(const SeqProb& P, WholeList& w, int lane, DeviceErr* err) {
  w.round = 0;
  w.pairs = w.most = 0;
  if (P.n_seqs > LPT_SEQS) return;
#pragma unroll
  for (int k = 0; k < LPT_SEQS / 32; ++k) {
    const int i = lane + 32 * k;
    w.it[k] = Items<KIND_MANY>{};
    if (i >= P.n_seqs) continue;
    w.it[k] = items_of<KIND_MANY>(P, false, seq_info(P, i, err));
    w.pairs += w.it[k].count;
    if (w.it[k].count > 0) w.most = max(w.most, w.it[k].tiles(w.it[k].count - 1));
  }
  w.pairs = __reduce_add_sync(0xffffffffu, w.pairs);
  w.most = __reduce_max_sync(0xffffffffu, w.most);
}
// Pair p of the list, by key tiles descending: its sequence and place there.
__device__ __forceinline__ void find_pair(const WholeList& w, int p, int lane, int& seq, int& u) {
  auto count = [&](int T) {
    int n = 0;
#pragma unroll
    for (int k = 0; k < LPT_SEQS / 32; ++k) n += pairs_from(w.it[k], T);
    return (int)__reduce_add_sync(0xffffffffu, n);
  };
  int lo = 1, hi = w.most;              // the largest T with more than p pairs of T tiles or more
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (count(mid) > p) lo = mid; else hi = mid - 1;
  }
  int left = p - count(lo + 1);
#pragma unroll
  for (int k = 0; k < LPT_SEQS / 32; ++k) {
    const int more = pairs_from(w.it[k], lo + 1), here = pairs_from(w.it[k], lo) - more;
    int incl = here;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += x;
    }
    const uint32_t found = __ballot_sync(0xffffffffu, left >= incl - here && left < incl);
    if (found != 0) {
      const int from = __ffs(found) - 1;
      seq = from + 32 * k;
      u = __shfl_sync(0xffffffffu, w.it[k].count - more - here + left - (incl - here), from);
      left = NO_TILE;                   // in no later run
    }
    const int all = __shfl_sync(0xffffffffu, incl, 31);
    if (left != NO_TILE) left -= all;
  }
}
__device__ __forceinline__ void next_item(const SeqProb& P, WholeList& w, Seg& g, WsHeader* hdr, int lane) {
  const int per = 2 * P.TQ;
  while (true) {
    unsigned item = blockIdx.x;
    if (w.round > 0) {
      if (lane == 0) item = gridDim.x + atomicAdd(&hdr->ticket, 1u);
      item = __shfl_sync(0xffffffffu, item, 0);
    }
    ++w.round;
    g.stop = item >= (P.n_seqs > LPT_SEQS ? P.items : (long long)w.pairs * P.Hkv);
    if (g.stop) return;
    const int pr = item / (unsigned)P.Hkv;
    g.kvh = item - pr * P.Hkv;
    int seq = 0, u;
    if (P.n_seqs > LPT_SEQS) {
      // sequence i's pairs lie at cu_q[i] / per + i and on (never more than
      // the gap to the next sequence's first)
      const int back = (int)(P.items / P.Hkv) - 1 - pr;
      int hi = P.n_seqs - 1;
      while (seq < hi) {
        const int mid = (seq + hi + 1) >> 1;
        if (P.cu_q[mid] / per + mid <= back) seq = mid; else hi = mid - 1;
      }
      u = back - (P.cu_q[seq] / per + seq);
    } else {
      find_pair(w, pr, lane, seq, u);
    }
    const SeqInfo s = seq_info(P, seq, &hdr->err);
    if (u < 0 || u >= ceil_div(s.Lq, per)) continue;
    g.lead = 0;
    g.row = s.row;
    g.q0 = s.q0;
    g.tok = u * per;
    g.ntok = min(per, s.Lq - g.tok);
    g.key0 = P.paged ? P.shared : s.k0;
    g.len = s.len;
    g.off = s.off;
    g.out = OUT_FINAL;
    g.slot = 0;
    fill_counts(P, g, 0, 1 << 30);
    return;
  }
}

// Split keys: the next part of this CTA's share.
__device__ __forceinline__ void next_part(const SeqProb& P, const SharePlan& plan, ShareWalk<KIND_MANY>& w, Seg& g, DeviceErr* err) {
  SharePart p;
  g.stop = !next_share_part(P, plan, w, p, err);
  if (g.stop) return;
  g.lead = p.lead;
  g.kvh = p.kvh;
  g.tok = p.item * 2 * P.TQ;
  g.ntok = min(2 * P.TQ, p.tokens - g.tok);
  g.row = p.lead ? plan.lead_row : w.s.row;
  g.q0 = p.lead ? 0 : w.s.q0;
  g.key0 = p.lead ? 0 : P.paged ? P.shared : w.s.k0;
  g.len = p.lead ? min(P.shared, plan.lead_len) : w.s.len;
  g.off = p.lead ? 0 : w.s.off;
  g.slot = p.slot;
  g.out = p.out;
  if (p.out == OUT_SLOT && (p.slot & 1)) P.many.split[blockIdx.x] = {p.parts, g.q0 + g.tok, g.ntok, g.kvh};
  fill_counts(P, g, p.t0, p.t1);
}

// V row `row` of a tile, which holds key `key` of the region: cleared past the
// region's end; where some row of the queries does not see it (key >=
// seen_by_all), its non-finite elements are replaced by zero and the tile is
// noted.  Returns whether it wrote.
template <bool BF16>
__device__ __forceinline__ bool repair_v_row(uint8_t* vt, int row, int key, int len, int seen_by_all, int* nf, int tile) {
  if (key < seen_by_all) return false;
  // 16-byte pieces, rows starting at different ones: no bank conflicts
  auto piece = [&](int c) { return reinterpret_cast<uint4*>(vt + (c >> 3) * 16384 + row * 128) + ((c + row) & 7); };
  if (key >= len) {
#pragma unroll
    for (int c = 0; c < 16; ++c) *piece(c) = make_uint4(0, 0, 0, 0);
    return true;
  }
  // an exponent of all ones, plus one, carries into the sign's place
  constexpr uint32_t E = BF16 ? 0x7F807F80u : 0x7C007C00u, ONE = BF16 ? 0x00800080u : 0x04000400u;
  uint32_t carry = 0;
#pragma unroll
  for (int c0 = 0; c0 < 16; c0 += 8) {
    uint4 w[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) w[c] = *piece(c0 + c);
#pragma unroll
    for (int c = 0; c < 8; ++c)
      carry |= ((w[c].x & E) + ONE) | ((w[c].y & E) + ONE) | ((w[c].z & E) + ONE) | ((w[c].w & E) + ONE);
  }
  if ((carry & 0x80008000u) == 0) return false;
  atomicMin(nf, tile);
  __threadfence_block();
#pragma unroll 1
  for (int c = 0; c < 16; ++c) {
    uint4 v = *piece(c);
    uint32_t* x = reinterpret_cast<uint32_t*>(&v);
    for (int e = 0; e < 4; ++e) {
      if (nonfinite16<BF16>(x[e])) x[e] &= 0xffff0000u;
      if (nonfinite16<BF16>(x[e] >> 16)) x[e] &= 0xffffu;
    }
    *piece(c) = v;
  }
  return true;
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

  dependents_may_start();
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
      mbar_init(&bar[B_QFULL + i], 1);
      mbar_init(&bar[B_QEMPTY + i], 1);
    }
    for (int i = 0; i < SEGS; ++i) {
      mbar_init(&bar[B_SEGFULL + i], 1);
      mbar_init(&bar[B_SEGEMPTY + i], SEG_READERS);
    }
    mi->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(&mi->tmem, 512);
    tmem_relinquish();
  }
  if (P.split) plan_shares<KIND_MANY, NUM_THREADS>(P, mi->plan, err);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = mi->tmem;
  if (warp < 8) {
    regs_inc<SOFTMAX_REGS>();
  } else {
    regs_dec<ISSUE_REGS>();
  }
  const Waits waits{bar, abort_flag, limit_ns, err};
  auto wait_all = [&](int b, uint32_t parity, uint32_t site) { return wait_warp(waits, b, parity, site); };

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
    const int rtok = over_G(P, r), rhead = r - rtok * P.G;
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
      // this row's limit, and the smallest of the tile's (the same in its four
      // warps; of both tiles' in the shared region, where limits do not ascend)
      const int t0 = g.tok + X * P.TQ, t1 = min(t0 + P.TQ, g.tok + g.ntok);
      int lim, gmin;
      if (g.lead) {
        lim = row_limit(P, 1, 0, g.len, min(tt, t1 - 1));
        gmin = g.len;
        for (int t = g.tok + lane; t < g.tok + g.ntok; t += 32) gmin = min(gmin, row_limit(P, g.lead, g.off, g.len, t));
        gmin = __reduce_min_sync(0xffffffffu, gmin);
      } else {
        lim = row_limit(P, 0, g.off, g.len, min(tt, t1 - 1));
        gmin = row_limit(P, g.lead, g.off, g.len, t0);
      }
      const bool active = __any_sync(0xffffffffu, valid);
      float m = -INFINITY, l = 0.0f;
      bool ok = true;
      for (int t = 0; t < n; ++t) {
        const int key = (g.tile0 + t) * KEYS;
        // S(t) has landed -- and with it P.V(t-1)
        if (!(ok = wait_all(B_SFULL + X, s_phase & 1, 0x4102))) break;
        ++s_phase;
        if (gmin < key + KEYS && (X == 0 || t >= g.n[0])) {
          // a tile that some row sees in part: this warp's 32 V rows.  Tile A's
          // warps do it where A has the tile: B's gmin is not below A's, and B's
          // product comes after A's, which waits for these warps' P.  So no
          // product reads V while it changes.
          const int ring = g.ring + t;
          if (!(ok = wait_all(B_VFULL + ring % STAGES, (ring / STAGES) & 1, 0x4103))) break;
          uint8_t* vt = sm + Smem::V + (ring % STAGES) * 32768;
          const int vr = 32 * wq + lane;
          if (repair_v_row<BF16>(vt, vr, key + vr, g.len, gmin, &mi->nf_tile[k % SEGS], g.tile0 + t))
            fence_async_smem();   // the products read it
          __syncwarp();
        }
        if (active) {
          tc_fence_after();
          uint32_t s[128];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(tS + 32 * c, s + 32 * c);
          tmem_wait_ld();
          const int nvalid = lim - key;   // keys of the tile that this row sees
          if (gmin < key + KEYS) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {   // bit e: key 32 c + e is seen
              const uint32_t bits = nvalid >= 32 * c + 32 ? 0xffffffffu : ~(0xffffffffu << max(0, nvalid - 32 * c));
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if ((bits >> e & 1u) == 0) s[32 * c + e] = 0xFF800000u;   // -inf: out of the max and the sum
            }
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
      const bool store = valid && in_bounds(row_inside(P, P.many, g.out, g.slot, token, head, X * 128 + r, SLOT_ROWS), err, 0x4105);
      const int nf = *reinterpret_cast<volatile int*>(&mi->nf_tile[k % SEGS]);
      const RowOut out = row_out(P, P.many, g.out, g.slot, store ? token : 0, store ? head : 0, X * 128 + r);
      if (store && out.lse != nullptr) *out.lse = g.out == OUT_FINAL ? lse2 * LN2 : lse2;
      // A row per lane would touch 32 lines with every store.  64 bytes of each
      // row go through shared memory instead (pieces XORed with the row pair: no
      // bank conflicts), and four lanes write a row: eight rows per store.
      uint8_t* const mine = out.h != nullptr ? out.h : reinterpret_cast<uint8_t*>(out.f);
      uint8_t* dst[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int from = 8 * i + (lane >> 2);
        const unsigned long long p = __shfl_sync(0xffffffffu, store ? (unsigned long long)(uintptr_t)mine : 0ull, from);
        dst[i] = reinterpret_cast<uint8_t*>((uintptr_t)p);
      }
      uint4* const stage = reinterpret_cast<uint4*>(sm + Smem::STAGE) + warp * 128;
      auto put = [&](const uint32_t* words, int off) {   // 16 words of every row, to byte `off` of it
#pragma unroll
        for (int p = 0; p < 4; ++p)
          stage[lane * 4 + (p ^ ((lane >> 1) & 3))] = make_uint4(words[4 * p], words[4 * p + 1], words[4 * p + 2], words[4 * p + 3]);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int from = 8 * i + (lane >> 2);
          const uint4 v = stage[from * 4 + ((lane & 3) ^ ((from >> 1) & 3))];
          if (dst[i] != nullptr) *reinterpret_cast<uint4*>(dst[i] + off + 16 * (lane & 3)) = v;
        }
        __syncwarp();
      };
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
          float z[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) z[e] = y[e];
          add_nonfinite<BF16, 32>(P, {g.key0, g.row, g.kvh}, nf * KEYS, min(lim, (g.tile0 + n) * KEYS), 32 * c, z);
#pragma unroll
          for (int e = 0; e < 32; ++e) y[e] = z[e];
        }
        uint32_t words[32];
        if (g.out == OUT_FINAL) {
#pragma unroll
          for (int e = 0; e < 16; ++e) words[e] = pack2<BF16>(y[2 * e], y[2 * e + 1]);
          put(words, 64 * c);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) words[e] = __float_as_uint(y[e]);
          put(words, 128 * c);
          put(words + 16, 128 * c + 64);
        }
      }
      tc_fence_before();   // O has been read: the next segment's first P.V follows this row's next P
      free_segment(k);
    }
  } else if (warp == 8) {
    // ------------------------------------------------------------ segment list
    WholeList whole;
    if (!P.split) start_list(P, whole, lane, err);
    const int ahead = P.split ? SEGS : 2;   // whole items: no further than needed, others may come to them first
    ShareWalk<KIND_MANY> w;
    if (P.split) {
      start_walk(P, mi->plan, w);
      if (lane == 0) P.many.split[blockIdx.x].parts = 0;
      __syncwarp();
    }
    int ring = 0, q0 = 0, q1 = 0;
    Seg g;
    for (int k = 0;; ++k) {
      if (k >= ahead && !wait_all(B_SEGEMPTY + (k - ahead) % SEGS, ((k - ahead) / SEGS) & 1, 0x4201)) break;
      if (P.split) next_part(P, mi->plan, w, g, err);
      else next_item(P, whole, g, hdr, lane);
      g.ring = ring;
      g.qidx[0] = q0;
      g.qidx[1] = q1;
      if (lane == 0) {
        mi->seg[k % SEGS] = g;
        mi->nf_tile[k % SEGS] = NO_TILE;
        __threadfence_block();
        mbar_arrive(&bar[B_SEGFULL + k % SEGS]);
      }
      __syncwarp();
      if (g.stop) break;
      ring += g.nload;
      q0 += g.n[0] > 0;
      q1 += g.n[1] > 0;
    }
    if (!P.split && P.n_seqs > LPT_SEQS) {   // sequences that the list passed by are looked at too, for what they report
      for (int i = blockIdx.x * 32 + lane; i < P.n_seqs; i += gridDim.x * 32) seq_info(P, i, err);
    }
    if (!P.split && lane == 0) {   // no CTA takes a ticket after its last: the last one out sets them back
      __threadfence();
      if (atomicAdd(&hdr->leaving, 1u) == gridDim.x - 1) {
        hdr->ticket = 0;
        hdr->leaving = 0;
      }
    }
  } else if (warp == 11) {
    // ------------------------------------------------------------ copies
    if (lane == 0) {
      asm volatile("prefetch.tensormap [%0];" ::"l"(&mq) : "memory");
      asm volatile("prefetch.tensormap [%0];" ::"l"(&mk) : "memory");
      asm volatile("prefetch.tensormap [%0];" ::"l"(&mv) : "memory");
    }
    // lane = (K or V, half of the channels, page of the tile)
    const int box_half = (lane >> 3) & 1, box_page = lane & 7;
    const CUtensorMap* map = lane < 16 ? &mk : &mv;
    uint8_t* const base = sm + (lane < 16 ? Smem::K : Smem::V) + box_half * 16384;
    const int full = lane < 16 ? B_KFULL : B_VFULL;
    int ring = 0, qn[2] = {0, 0};
    bool ok = true;
    for (int k = 0; ok; ++k) {
      const Seg* seg = segment(k, 0x4203);
      if (!(ok = seg != nullptr) || seg->stop) break;
      const Seg& g = *seg;
      const int nload = g.nload, len = g.len, key0 = g.key0, kvh = g.kvh;
#pragma unroll
      for (int X = 0; X < 2; ++X) {
        if (!ok || (X ? g.n[1] : g.n[0]) == 0) continue;
        const int c = qn[X];
        if (c > 0 && !(ok = wait_all(B_QEMPTY + X, (c - 1) & 1, 0x4202))) continue;
        if (lane == 0) {
          mbar_expect_tx(&bar[B_QFULL + X], 2u * 128u * P.G * P.TQ);
          for (int h = 0; h < 2; ++h)
            tma_load4(sm + (X ? Smem::QB : Smem::QA) + h * 16384, &mq, 64 * h, 0, kvh, g.q0 + g.tok + X * P.TQ,
                      &bar[B_QFULL + X]);
        }
        __syncwarp();
        ++qn[X];
      }
      if (!ok) break;
      const int* trow = P.paged ? P.table + (long long)g.row * P.max_pages : nullptr;
      // this lane's page of tile t; -1: none
      auto page_of = [&](int t) {
        const int first = (g.tile0 + t) * KEYS + (box_page << P.page_shift);
        if (t >= nload || box_page >= KEYS >> P.page_shift || first >= len) return -1;
        if (!in_bounds(g.row >= 0 && g.row < P.max_seqs && (key0 + first) >> P.page_shift < P.max_pages, err, 0x4210))
          return P.n_pages;
        const int page = trow[(key0 + first) >> P.page_shift];
        if ((uint32_t)page < (uint32_t)P.n_pages) return page;
        report(err, DEVERR_BOUNDS, 0x4204);   // not a page: read as zeros
        return P.n_pages;
      };
      int page = P.paged ? page_of(0) : -1;
      for (int t = 0; t < nload; ++t, ++ring) {
        const int st = ring % STAGES;
        const uint32_t parity = ((ring / STAGES) - 1) & 1;
        const int next = P.paged ? page_of(t + 1) : -1;
        const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, page >= 0));   // four per page
        if (ring >= STAGES && !(ok = wait_all(B_KEMPTY + st, parity, 0x4205))) break;
        const uint32_t bytes = P.paged ? boxes * 64u * P.page_size : 32768u;
        if (lane == 0) mbar_expect_tx(&bar[B_KFULL + st], bytes);
        __syncwarp();
        auto issue = [&] {
          if (P.paged) {
            if (page >= 0)
              tma_load4(base + st * 32768 + ((box_page << P.page_shift) * 128), map, 64 * box_half, 0, kvh, page,
                        &bar[full + st]);
          } else if (box_page == 0) {
            tma_load4(base + st * 32768, map, 64 * box_half, 0, kvh, key0 + (g.tile0 + t) * KEYS, &bar[full + st]);
          }
        };
        if (lane < 16) issue();
        __syncwarp();
        if (ring >= STAGES && !(ok = wait_all(B_VEMPTY + st, parity, 0x4206))) break;
        if (lane == 0) mbar_expect_tx(&bar[B_VFULL + st], bytes);
        __syncwarp();
        if (lane >= 16) issue();
        __syncwarp();
        page = next;
      }
      free_segment(k);
    }
    // every copy lands before the CTA exits, also after another role gave up
    for (int X = 0; X < 2; ++X)
      if (qn[X] > 0) mbar_wait(&bar[B_QFULL + X], (qn[X] - 1) & 1, limit_ns, err, 0x4207);
    for (int t = ring > STAGES ? ring - STAGES : 0; t < ring; ++t) {
      mbar_wait(&bar[B_KFULL + t % STAGES], (t / STAGES) & 1, limit_ns, err, 0x4208);
      mbar_wait(&bar[B_VFULL + t % STAGES], (t / STAGES) & 1, limit_ns, err, 0x4209);
    }
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
    uint32_t p_phase[2] = {0, 0};
    int turn = 0;                  // groups of this tile so far
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
      const int q = __shfl_sync(0xffffffffu, X ? g.qidx[1] : g.qidx[0], 0);
      const int stop = __shfl_sync(0xffffffffu, g.stop, 0);
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
          if (t == n - 1) umma_commit(&bar[B_QEMPTY + X]);
        }
        __syncwarp();
      };
      if (n > 0 && !(ok = wait_all(B_QFULL + X, q & 1, 0x4304))) break;
      if (!(ok = k_full(0))) break;
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
          if (!(ok = wait_all(B_TURN + X, (X ? turn : turn - 1) & 1, 0x4306))) break;
        }
        ++turn;
        if (t < n) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {   // O += P(t) V(t), P from TMEM
            if (!ok || !(ok = wait_all(B_PFULL + 2 * half + X, p_phase[half], 0x4305))) continue;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int kk = 4 * half; kk < 4 * half + 4; ++kk)
                umma_f16_tmem_a(tO, tS + 64 + 8 * kk, vt + kk * (2048 >> 4), IDESC_PV, (t > 0) || (kk > 0));
            }
            __syncwarp();
          }
          if (!ok) break;
          p_phase[0] ^= 1u;
          p_phase[1] ^= 1u;
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

// ---------------------------------------------------------------- join
// o = sum_s 2^(lse_s - M) o_s / sum_s 2^(lse_s - M),  M = max lse_s, over the
// partial results of a row: one warp per row, four channels per lane.
// Memory-bound: reads 516 bytes per part and row, writes 256.
struct Parts {           // part c lies at first + c step (+ back for c = 0)
  const float *o, *l;
  long long first, step, back;
  int n;
  long long rows;      // of the buffer
};
__device__ __forceinline__ Parts slot_parts(const ShareBuf& b, int slot_rows, int cta, int n, int row) {
  // the item goes on behind the first CTA's share (slot 1), began before the others' (slot 0)
  return {b.slot_o, b.slot_lse, 2ll * cta * slot_rows + row, 2ll * slot_rows, slot_rows, n, 2ll * b.grid * slot_rows};
}
template <bool BF16>
__device__ __forceinline__ void join_row(const SeqProb& P, const Parts& a, const Parts& b, int token, int head, int lane) {
  float M = -INFINITY, sum = 0.0f;
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  const int n = a.n + b.n;
  // four parts at a time, all their loads before the first use
  for (int c0 = 0; c0 < n; c0 += 4) {
    float l[4];
    float4 x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      l[k] = -INFINITY;
      x[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      const int c = c0 + k;
      if (c >= n) continue;
      const Parts& p = c < a.n ? a : b;
      const int d = c < a.n ? c : c - a.n;
      const long long at = p.first + d * p.step + (d == 0 ? p.back : 0);
      if (!in_bounds(at >= 0 && at < p.rows, P.err, 0x4601)) continue;
      l[k] = p.l[at];
      x[k] = reinterpret_cast<const float4*>(p.o + at * D)[lane];
    }
    const float m = fmaxf(fmaxf(M, fmaxf(l[0], l[1])), fmaxf(l[2], l[3]));
    if (l[0] == -INFINITY && l[1] == -INFINITY && l[2] == -INFINITY && l[3] == -INFINITY) continue;   // saw no key
    const float old = exp2f(M - m);
    M = m;
    sum *= old;
    acc = make_float4(acc.x * old, acc.y * old, acc.z * old, acc.w * old);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float w = exp2f(l[k] - m);             // NaN stays NaN
      sum += w;
      acc.x = fmaf(w, x[k].x, acc.x);
      acc.y = fmaf(w, x[k].y, acc.y);
      acc.z = fmaf(w, x[k].z, acc.z);
      acc.w = fmaf(w, x[k].w, acc.w);
    }
  }
  if (!in_bounds(token >= 0 && token < P.total_q && head >= 0 && head < P.Hq, P.err, 0x4602)) return;
  const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
  const uint2 out = make_uint2(pack2<BF16>(acc.x * inv, acc.y * inv), pack2<BF16>(acc.z * inv, acc.w * inv));
  *reinterpret_cast<uint2*>(P.o + token * P.o_tok + head * P.o_head + 8 * lane) = out;
  if (lane == 0 && P.lse != nullptr)
    P.lse[(long long)token * P.Hq + head] = sum != 0.0f ? (M + log2f(sum)) * LN2 : -INFINITY;
}

// No shared region: only the rows of items that were split, a CTA's slot per
// grid row, 8 rows of it per block; KIND_MANY's CTAs first.
template <bool BF16>
__global__ void __launch_bounds__(256) join_items_kernel(const __grid_constant__ SeqProb P) {
  wait_for_predecessor();
  const bool few = blockIdx.x >= P.many.grid * (SLOT_ROWS / 8);
  const ShareBuf& b = few ? P.few : P.many;
  const int slot_rows = few ? FEW_ROWS : SLOT_ROWS, blk = blockIdx.x - (few ? P.many.grid * (SLOT_ROWS / 8) : 0);
  const int cta = blk / (slot_rows / 8), row = blk % (slot_rows / 8) * 8 + (threadIdx.x >> 5);
  const SplitItem it = b.split[cta];
  if (it.parts == 0) return;
  // the row's token and head, if it has any
  const int r = few ? row : row & 127, t = over_G(P, r), gh = r - t * P.G;
  const int tt = few ? t : t + (row >> 7) * P.TQ;
  if ((!few && t >= P.TQ) || tt >= it.tokens) return;
  join_row<BF16>(P, slot_parts(b, slot_rows, cta, it.parts, row), Parts{}, it.token + tt, it.kvh * P.G + gh, threadIdx.x & 31);
}

// With a shared region: every row has a result of it and one of its own
// region, each whole or split.  A block takes P.join_heads heads of one token,
// whose sequence it looks up once.
template <int KIND>
struct RegionParts {
  long long first, all, share;   // first tile of the token's item at key head 0; units per key head
  int tiles, row0, lead;
  const ShareBuf* b;
  __device__ __forceinline__ void find(const SeqProb& P, const ShareBuf& buf, bool is_lead, const SeqInfo& s, int i, int token) {
    using K = Kind<KIND>;
    const Items<KIND> it = items_of<KIND>(P, is_lead, s);
    const int t = is_lead ? token : token - s.q0, per = K::tokens_per_item(P), u = t / per;
    b = &buf;
    lead = is_lead;
    share = share_of(buf.starts[P.n_seqs], buf.grid);
    all = it.all();
    first = (is_lead ? 0 : buf.starts[i]) + it.before(u) + K::W_ITEM;
    tiles = it.tiles(u);
    row0 = slot_row<KIND>(P, t - u * per, 0);
  }
  __device__ __forceinline__ Parts parts(const SeqProb& P, int kvh, int gh, long long row) const {
    using K = Kind<KIND>;
    const long long a = first + kvh * all;
    const int c0 = quotient(a, share), c1 = quotient(a + (long long)(tiles - 1) * K::TILE, share);
    if (c0 == c1) return {lead ? P.lead_o : P.own_o, lead ? P.lead_lse : P.own_lse, row, 0, 0, 1, (long long)P.total_q * P.Hq};
    return slot_parts(*b, K::SLOT, c0, c1 - c0 + 1, row0 + gh);
  }
};
template <bool BF16, int LEAD, int OWN>
__device__ __forceinline__ void join_token(const SeqProb& P, int token, int h0, const SeqInfo& s, int i) {
  RegionParts<LEAD> lead;
  RegionParts<OWN> own;
  lead.find(P, LEAD == KIND_FEW ? P.few : P.many, true, s, i, token);
  own.find(P, OWN == KIND_FEW ? P.few : P.many, false, s, i, token);
  const int h1 = min(P.Hq, h0 + P.join_heads);
  for (int head = h0 + (threadIdx.x >> 5); head < h1; head += 8) {
    const int kvh = head / P.G, gh = head - kvh * P.G;
    const long long row = (long long)token * P.Hq + head;
    join_row<BF16>(P, lead.parts(P, kvh, gh, row), own.parts(P, kvh, gh, row), token, head, threadIdx.x & 31);
  }
}
template <bool BF16>
__global__ void __launch_bounds__(256) join_rows_kernel(const __grid_constant__ SeqProb P) {
  const int per_token = ceil_div(P.Hq, P.join_heads), token = blockIdx.x / per_token;
  const int h0 = (blockIdx.x - token * per_token) * P.join_heads;
  const int i = seq_of_token(P, token);
  const SeqInfo s = seq_info(P, i, nullptr);
  wait_for_predecessor();
  if (token < s.q0 || token >= s.q0 + s.Lq) return;   // behind the last sequence
  const bool lead_few = takes<KIND_FEW>(P, P.total_q), own_few = takes<KIND_FEW>(P, s.Lq);
  if (lead_few) join_token<BF16, KIND_FEW, KIND_FEW>(P, token, h0, s, i);
  else if (own_few) join_token<BF16, KIND_MANY, KIND_FEW>(P, token, h0, s, i);
  else join_token<BF16, KIND_MANY, KIND_MANY>(P, token, h0, s, i);
}

// The list warp waits for a segment to be finished, which over millions of keys
// takes longer than any other wait: each of the tiles it may have adds what the
// slowest ones take (6000 cycles at 1.1 GHz), with a margin.
uint64_t wait_limit_of(const SeqProb& p) {
  const long long keys = p.paged ? (long long)p.max_pages << p.page_shift : p.total_k;
  return wait_limit() + 8000ull * (uint64_t)(keys / KEYS + 1);
}

template <bool BF16>
cudaError_t launch(const SeqProb& p, const SeqMaps& m, void* ws,
                   cudaStream_t st) {
  cudaError_t e;
  if (p.many.grid > 0) {
    const int smem = Smem::BYTES + 1024;   // > half the SM: one CTA per SM owns all 512 TMEM columns
    auto kern = seq_attn_kernel<BF16>;
    static OncePerDevice once;
    e = once.run([&] {
      cudaError_t r = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      cudaFuncAttributes fa;   // the setmaxnreg split needs exactly LAUNCH_REGS at launch
      if (r == cudaSuccess) r = cudaFuncGetAttributes(&fa, kern);
      return r == cudaSuccess && fa.numRegs != LAUNCH_REGS ? cudaErrorInvalidConfiguration : r;
    });
    if (e != cudaSuccess) return e;
    e = launch_after(false, kern, p.many.grid, NUM_THREADS, smem, st, p, m.q, m.k, m.v, static_cast<WsHeader*>(ws),
                     wait_limit_of(p));
    if (e != cudaSuccess) return e;
  }
  if (p.few.grid > 0 && (e = launch_few_attention(p, static_cast<WsHeader*>(ws), p.many.grid > 0, st)) != cudaSuccess) return e;
  if (!p.split) return cudaSuccess;
  if (p.shared == 0)
    return launch_after(true, join_items_kernel<BF16>, p.many.grid * (SLOT_ROWS / 8) + p.few.grid * (FEW_ROWS / 8), 256, 0, st, p);
  return launch_after(true, join_rows_kernel<BF16>, (unsigned)p.total_q * ceil_div(p.Hq, p.join_heads), 256, 0, st, p);
}

}  // namespace

cudaError_t launch_seq_attention(const SeqProb& p, const SeqMaps& m, void* ws, cudaStream_t st) {
  return p.bf16 ? launch<true>(p, m, ws, st) : launch<false>(p, m, ws, st);
}

}  // namespace ra
