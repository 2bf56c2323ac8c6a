// ra_serve.h -- problem and launch interface of the packed-prompt attention
// and the paged-cache attention (ra_packed.cu), shared with the C ABI
// (ra_serve_api.cu).
#pragma once
#include <cuda.h>

#include "ra_internal.h"

namespace ra {

constexpr int KEYS = 128;        // keys per tile
constexpr int SLOT_ROWS = 256;   // query rows of a work item: two 128-row tiles

// One attention call over sequences whose query tokens are packed: sequence i
// owns tokens [q0, q0 + Lq).  Keys are either packed rows (paged = 0) or the
// pages of a cache (paged = 1), there in two regions: the first `shared`
// tokens, taken from one sequence for the whole batch, and each sequence's
// own tokens behind them.
struct SeqProb {
  int n_seqs, Hq, Hkv;
  int G;                         // query heads per key head
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
  int split;                     // 1: equal shares of key tiles per CTA, joined afterwards; 0: whole items
  int grid;
  long long items;               // split = 0: upper bound of work items
  long long* starts;             // split: first own tile of each sequence, [n_seqs + 1]
  float *slot_o, *slot_lse;      // split: [grid][2][SLOT_ROWS](x 128)
  float *lead_o, *lead_lse;      // shared > 0: [total_q * Hq](x 128), the shared region's result
  float *own_o, *own_lse;        // shared > 0: the own region's result
};

// Workspace of a split call (after the 256-byte header).
struct SeqWs {
  size_t starts, slot_o, slot_lse, lead_o, lead_lse, own_o, own_lse, total;
};
inline SeqWs seq_ws(int n_seqs, long long total_q, int Hq, int shared, int grid) {
  SeqWs L;
  size_t o = align256(sizeof(WsHeader));
  const size_t rows = (size_t)total_q * Hq, slots = (size_t)grid * 2 * SLOT_ROWS;
  L.starts = o;
  o = align256(o + sizeof(long long) * ((size_t)n_seqs + 1));
  L.slot_o = o;
  o = align256(o + slots * D * sizeof(float));
  L.slot_lse = o;
  o = align256(o + slots * sizeof(float));
  L.lead_o = o;
  if (shared) o = align256(o + rows * D * sizeof(float));
  L.lead_lse = o;
  if (shared) o = align256(o + rows * sizeof(float));
  L.own_o = o;
  if (shared) o = align256(o + rows * D * sizeof(float));
  L.own_lse = o;
  if (shared) o = align256(o + rows * sizeof(float));
  L.total = o;
  return L;
}

cudaError_t launch_seq_attention(const SeqProb& p, const CUtensorMap& mq, const CUtensorMap& mk,
                                 const CUtensorMap& mv, void* ws, cudaStream_t st);

}  // namespace ra
