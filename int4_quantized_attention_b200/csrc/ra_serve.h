// ra_serve.h -- problem and launch interface of the packed-prompt attention
// and the paged-cache attention (ra_packed.cu), shared with the C ABI
// (ra_serve_api.cu).
#pragma once
#include <cuda.h>

#include "ra_internal.h"

namespace ra {

constexpr int KEYS = 128;        // keys per tile
constexpr int FEW_ROWS = 64;     // paged items of at most this many rows run on the warp-level MMA
constexpr int FEW_KEYS = 64;     // keys per tile there
constexpr int FEW_CTAS = 3;      // and CTAs per SM
constexpr int SLOT_ROWS = 256;   // query rows of a work item: two 128-row tiles

// One attention call over sequences whose query tokens are packed: sequence i
// owns tokens [q0, q0 + Lq).  Keys are either packed rows (paged = 0) or the
// pages of a cache (paged = 1), there in two regions: the first `shared`
// tokens, taken from one sequence for the whole batch, and each sequence's
// own tokens behind them.
struct SplitItem;

// One kernel's shares of the key tiles (split calls).
struct ShareBuf {
  int grid;                      // CTAs; 0: not launched
  long long* starts;             // first unit of each sequence, [n_seqs + 1]
  float *slot_o, *slot_lse;      // [grid][2][rows of a slot](x 128)
  SplitItem* split;              // [grid], the item that goes on behind each share
};

struct SeqProb {
  int n_seqs, Hq, Hkv;
  int G;                         // query heads per key head
  uint32_t inv_G;                // ceil(2^16 / G)
  int TQ;                        // tokens per 128-row tile: 128 / G
  int total_q, total_k;
  int causal;
  int bf16;
  float cs;                      // softmax scale * log2(e)
  const int *cu_q, *cu_k;        // [n_seqs + 1]; cu_q NULL: one token per sequence
  int paged, shared;
  int page_size, page_shift, max_pages, n_pages, max_seqs;
  const int *seqs, *lens, *table;
  const uint8_t* v;              // for the rare repair of non-finite values
  long long v_tok, v_head;       // byte strides of v (paged: within a page; v_page between pages)
  long long v_page;
  uint8_t* o;
  long long o_tok, o_head;       // byte strides
  float* lse;                    // [total_q][Hq] or NULL
  const uint8_t* q;              // for the kernel of few rows: byte strides
  long long q_tok, q_head;
  const uint8_t* k;              // paged: as v
  int split;                     // 1: equal shares of key tiles per CTA, joined afterwards; 0: whole items
  long long items;               // split = 0: upper bound of work items
  int join_heads;                // heads per block of the join by rows
  int lead_only;                 // the kernel of many rows has the shared region alone
  ShareBuf many, few;            // the two kernels' shares
  float *lead_o, *lead_lse;      // shared > 0: [total_q * Hq](x 128), the shared region's result
  float *own_o, *own_lse;        // shared > 0: the own region's result
  DeviceErr* err;                // for the joins' self-checks
};

// Workspace of a split call (after the 256-byte header).
struct SeqWs {
  size_t many_starts, many_split, many_o, many_lse, few_starts, few_split, few_o, few_lse, lead_o, lead_lse, own_o, own_lse, total;
};
inline SeqWs seq_ws(int n_seqs, long long total_q, int Hq, int shared, int many, int few) {
  SeqWs L;
  size_t o = align256(sizeof(WsHeader));
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = align256(o + bytes);
    return at;
  };
  const size_t rows = shared ? (size_t)total_q * Hq : 0, starts = sizeof(long long) * ((size_t)n_seqs + 1);
  const size_t many_rows = (size_t)many * 2 * SLOT_ROWS, few_rows = (size_t)few * 2 * FEW_ROWS;
  L.many_starts = take(many ? starts : 0);
  L.many_split = take(16 * (size_t)many);
  L.many_o = take(many_rows * D * sizeof(float));
  L.many_lse = take(many_rows * sizeof(float));
  L.few_starts = take(few ? starts : 0);
  L.few_split = take(16 * (size_t)few);
  L.few_o = take(few_rows * D * sizeof(float));
  L.few_lse = take(few_rows * sizeof(float));
  L.lead_o = take(rows * D * sizeof(float));
  L.lead_lse = take(rows * sizeof(float));
  L.own_o = take(rows * D * sizeof(float));
  L.own_lse = take(rows * sizeof(float));
  L.total = o;
  return L;
}

// Tensor maps of the call.
struct SeqMaps {
  CUtensorMap q, k, v;
};

cudaError_t launch_few_attention(const SeqProb& p, WsHeader* hdr, bool overlap, cudaStream_t st);
cudaError_t launch_seq_attention(const SeqProb& p, const SeqMaps& m, void* ws, cudaStream_t st);

}  // namespace ra
