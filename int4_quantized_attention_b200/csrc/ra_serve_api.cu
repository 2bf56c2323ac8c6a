// ra_serve_api.cu -- host side of the packed-sequence and paged-cache calls of
// include/rotate_attn.h: argument checks, tensor maps, workspaces and the
// choice between whole work items and split keys.  No allocation.
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include "ra_cache.h"
#include "ra_serve.h"

namespace {

using ra::align256;

ra_status fail(ra_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
ra_status fail(ra_status s, const char* fmt, ...) {
  char msg[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof(msg), fmt, ap);
  va_end(ap);
  ra::set_error_detail(msg);
  return s;
}

ra_status cuda_fail(cudaError_t e, const char* what) {
  cudaGetLastError();
  return fail(RA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned(const void* p, uintptr_t n) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// ---------------------------------------------------------------- tensor maps
typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                             const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                             CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encoder() {
  static EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      return (EncodeFn) nullptr;
    }
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}

// A 16-bit tensor of 128 channels x three outer dimensions (strides in
// bytes), copied in boxes of 64 channels with the 128-byte swizzle.
bool make_map(CUtensorMap* m, int bf16, const void* base, const cuuint64_t (&outer)[3], const cuuint64_t (&stride)[3],
              const cuuint32_t (&box)[3]) {
  const EncodeFn fn = encoder();
  if (fn == nullptr) return false;
  const cuuint64_t dims[4] = {128, outer[0], outer[1], outer[2]};
  const cuuint64_t strides[3] = {stride[0], stride[1], stride[2]};
  const cuuint32_t boxes[4] = {64, box[0], box[1], box[2]}, ones[4] = {1, 1, 1, 1};
  return fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<void*>(base),
            dims, strides, boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// ---------------------------------------------------------------- checks
ra_status check_heads(int Hq, int Hkv, int d) {
  if (d != ra::D) return fail(RA_ERR_UNSUPPORTED, "head_dim %d: only 128 is built", d);
  if (Hq < 1 || Hkv < 1 || Hq % Hkv != 0) return fail(RA_ERR_INVALID_ARG, "Hq = %d is not a multiple of Hkv = %d", Hq, Hkv);
  if (Hq / Hkv > 128) return fail(RA_ERR_UNSUPPORTED, "%d query heads per key head: at most 128", Hq / Hkv);
  if (Hq > 65535) return fail(RA_ERR_UNSUPPORTED, "Hq = %d: at most 65535", Hq);
  return RA_OK;
}

// A stride of a dimension of n entries: 16-byte steps that a tensor map takes.
bool stride_ok(long long s, long long n) {
  return n <= 1 || (s >= ra::D && s % 8 == 0 && s < (1ll << 38));
}
ra_status check_strides(const char* name, long long tok, long long head, long long tokens, int heads) {
  if (!stride_ok(tok, tokens) || !stride_ok(head, heads))
    return fail(RA_ERR_INVALID_ARG, "%s strides (%lld, %lld): multiples of 8 elements from 128 on", name, tok, head);
  return RA_OK;
}
ra_status check_out_strides(long long tok, long long head, long long tokens, int heads) {
  const ra_status st = check_strides("o", tok, head, tokens, heads);
  if (st != RA_OK) return st;
  if (tokens > 1 && heads > 1 && tok < (heads - 1) * head + ra::D && head < (tokens - 1) * tok + ra::D)
    return fail(RA_ERR_INVALID_ARG, "o's rows overlap (strides %lld, %lld)", tok, head);
  return RA_OK;
}
// A size-1 dimension's stride may be anything: what a tensor map gets for it.
cuuint64_t map_stride(long long s, long long n) { return n <= 1 ? 256 : (cuuint64_t)s * 2; }

ra_status check_scale(double scale) {
  const float c = (float)(scale * 1.4426950408889634);   // what the kernels multiply scores by
  if (!(scale >= 0.0) || !std::isfinite(c) || (scale > 0.0 && c == 0.0f))
    return fail(RA_ERR_INVALID_ARG, "softmax scale must be positive and finite (0: 1/sqrt(d))");
  return RA_OK;
}
float log2_scale(double scale) {
  return (float)((scale > 0.0 ? scale : 1.0 / std::sqrt((double)ra::D)) * 1.4426950408889634);
}

ra_status sm_count(int* out) {
  static std::atomic<int> known[64];   // per device; 0: not asked yet
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && dev < 64 && (*out = known[dev].load(std::memory_order_relaxed)) != 0) return RA_OK;
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(out, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess && dev < 64) known[dev].store(*out, std::memory_order_relaxed);
  return e == cudaSuccess ? RA_OK : cuda_fail(e, "device query");
}

// Workspace sizes are fixed without a device: at most this many SMs work on split keys.
constexpr int SM_BOUND = 148;

// ---------------------------------------------------------------- packed
// Upper bound of the work items of a packed call, from what the host knows.
long long packed_items(int total_q, int n_seqs, int TQ, int Hkv) {
  return ((long long)total_q / (2 * TQ) + n_seqs) * Hkv;
}
ra_status check_packed(const ra_packed* p) {
  if (p == nullptr) return fail(RA_ERR_INVALID_ARG, "problem is NULL");
  ra_status st = check_heads(p->Hq, p->Hkv, p->d);
  if (st != RA_OK) return st;
  if (p->n_seqs < 1) return fail(RA_ERR_INVALID_ARG, "n_seqs must be >= 1 (got %d)", p->n_seqs);
  if (p->dtype != RA_FP16 && p->dtype != RA_BF16) return fail(RA_ERR_INVALID_ARG, "dtype %d unknown", p->dtype);
  if (p->causal != 0 && p->causal != 1) return fail(RA_ERR_INVALID_ARG, "causal must be 0 or 1, not %d", p->causal);
  if (p->total_q < 0 || p->total_k < 0) return fail(RA_ERR_INVALID_ARG, "negative token count");
  if (p->total_q > (1 << 30) || p->total_k > (1 << 30) || p->n_seqs > (1 << 24))
    return fail(RA_ERR_UNSUPPORTED, "at most 2^30 tokens and 2^24 sequences");
  if (packed_items(p->total_q, p->n_seqs, 128 / (p->Hq / p->Hkv), p->Hkv) >= (1ll << 31))
    return fail(RA_ERR_UNSUPPORTED, "2^31 work items or more");
  if ((st = check_scale(p->scale)) != RA_OK) return st;
  if ((st = check_strides("q", p->q_token, p->q_head, p->total_q, p->Hq)) != RA_OK) return st;
  if ((st = check_strides("k", p->k_token, p->k_head, p->total_k, p->Hkv)) != RA_OK) return st;
  if ((st = check_strides("v", p->v_token, p->v_head, p->total_k, p->Hkv)) != RA_OK) return st;
  return check_out_strides(p->o_token, p->o_head, p->total_q, p->Hq);
}

// Few items leave SMs idle: split the keys instead. Below two items per SM equal shares mostly win or tie, above it
// their partial rows and the join cost more than the idle tail. Time on the GPU, split / whole items, bf16 and causal
// where nothing else is said: 2 chunks of 65-160 after 30000, 64/8 heads, 0.4 items per SM: 226 / 410 us; 4 of 300-400
// after 2000, 32/8, 1.3 items: 75 / 81; 2 of 1000-1500, 32/8, 2.2: 58 / 47; one of 4096 both ways, 24 heads, 2.6: 191 /
// 190; 3 of 1000-5000 both ways, 24 heads, 5.7: 374 / 364; one of 8192, 32/8, 6.9: 457 / 442; 13 of 40-2048, 32/8, 8.2:
// 147 / 134. Two calls of few items are the other way round: one of 2500 both ways, 24 heads (1.6 items, 100 / 88), and
// 5 texts of 1-77, 24 heads, fp16, which have one key tile each (0.8 items, 17 / 12).
bool packed_split(const ra_packed* p) {
  return packed_items(p->total_q, p->n_seqs, 128 / (p->Hq / p->Hkv), p->Hkv) < 2 * SM_BOUND;
}

// ---------------------------------------------------------------- cache
ra_status check_cache(const ra_cache_problem* p, ra::CacheProb* out) {
  if (p == nullptr) return fail(RA_ERR_INVALID_ARG, "cache problem is NULL");
  if (p->d != ra::D) return fail(RA_ERR_UNSUPPORTED, "head_dim %d: only 128 is built", p->d);
  if (p->dtype != RA_FP16 && p->dtype != RA_BF16) return fail(RA_ERR_INVALID_ARG, "dtype %d unknown", p->dtype);
  if (p->layers < 1 || p->n_pages < 1 || p->Hkv < 1 || p->max_seqs < 1 || p->max_pages < 1)
    return fail(RA_ERR_INVALID_ARG, "layers, n_pages, Hkv, max_seqs and max_pages must be >= 1");
  int shift = 4;
  while (shift < 8 && (1 << shift) != p->page_size) ++shift;
  if (shift == 8) return fail(RA_ERR_UNSUPPORTED, "page size %d: 16, 32, 64 or 128 tokens", p->page_size);
  if (p->layers > 65535 || p->Hkv > 65535) return fail(RA_ERR_UNSUPPORTED, "at most 65535 layers and key heads");
  if ((long long)p->max_seqs * p->max_pages >= (1ll << 31) || ((long long)p->max_pages << shift) >= (1ll << 30) ||
      p->n_pages > (1 << 24))
    return fail(RA_ERR_UNSUPPORTED, "table too large (max_seqs x max_pages < 2^31, max_pages x page_size < 2^30, "
                                    "n_pages <= 2^24)");
  const double bytes = 256.0 * p->layers * p->n_pages * p->Hkv * p->page_size;
  if (bytes >= 1099511627776.0) return fail(RA_ERR_UNSUPPORTED, "pool of 2^40 bytes or more");
  if (out) {
    out->layers = p->layers;
    out->n_pages = p->n_pages;
    out->page_size = p->page_size;
    out->page_shift = shift;
    out->Hkv = p->Hkv;
    out->max_seqs = p->max_seqs;
    out->max_pages = p->max_pages;
  }
  return RA_OK;
}

size_t half_pool(const ra_cache_problem* p) {
  return (size_t)256 * p->layers * p->n_pages * p->Hkv * p->page_size;
}

ra_status check_cache_call(const ra_cache_problem* p, const ra_cache* c, const void* ws, size_t bytes,
                           ra::CacheProb* out) {
  const ra_status st = check_cache(p, out);
  if (st != RA_OK) return st;
  if (c == nullptr || !aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->refs, 16) || !aligned(c->lens, 16) ||
      !aligned(c->table, 16))
    return fail(RA_ERR_INVALID_ARG, "a cache pointer is NULL or not 16-byte aligned");
  if (!aligned(ws, 256)) return fail(RA_ERR_INVALID_ARG, "workspace pointer NULL or not 256-byte aligned");
  const size_t need = ra::cache_ws(p->n_pages, p->max_seqs).total;
  if (bytes < need) return fail(RA_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", bytes, need);
  out->k = static_cast<uint8_t*>(c->k);
  out->v = static_cast<uint8_t*>(c->v);
  out->refs = c->refs;
  out->lens = c->lens;
  out->table = c->table;
  return RA_OK;
}
ra_status check_list(const void* list, int n, int max_seqs) {
  if (n < 0 || n > max_seqs) return fail(RA_ERR_INVALID_ARG, "list of %d rows: 0 to max_seqs = %d", n, max_seqs);
  if (n > 0 && !aligned(list, 4)) return fail(RA_ERR_INVALID_ARG, "a list is NULL or misaligned");
  return RA_OK;
}

ra_status check_attn(const ra_cache_problem* p, const ra_cache_attn* a) {
  ra_status st = check_cache(p, nullptr);
  if (st != RA_OK) return st;
  if (a == nullptr) return fail(RA_ERR_INVALID_ARG, "attention problem is NULL");
  if ((st = check_heads(a->Hq, p->Hkv, p->d)) != RA_OK) return st;
  if (a->n_seqs < 1) return fail(RA_ERR_INVALID_ARG, "n_seqs must be >= 1 (got %d)", a->n_seqs);
  if (a->total_q < 0) return fail(RA_ERR_INVALID_ARG, "negative token count");
  if (a->total_q > (1 << 30) || a->n_seqs > (1 << 24))
    return fail(RA_ERR_UNSUPPORTED, "at most 2^30 tokens and 2^24 sequences");
  if ((long long)a->total_q * a->Hq >= (1ll << 31)) return fail(RA_ERR_UNSUPPORTED, "2^31 query rows or more");
  if (a->layer < 0 || a->layer >= p->layers) return fail(RA_ERR_INVALID_ARG, "layer %d of %d", a->layer, p->layers);
  if (a->shared < 0 || a->shared % p->page_size != 0)
    return fail(RA_ERR_INVALID_ARG, "shared = %d is not a multiple of the page size %d", a->shared, p->page_size);
  if (a->shared > p->max_pages * p->page_size)
    return fail(RA_ERR_INVALID_ARG, "shared = %d: a row holds at most %d tokens", a->shared, p->max_pages * p->page_size);
  if ((st = check_scale(a->scale)) != RA_OK) return st;
  if ((st = check_strides("q", a->q_token, a->q_head, a->total_q, a->Hq)) != RA_OK) return st;
  return check_out_strides(a->o_token, a->o_head, a->total_q, a->Hq);
}

void fill_common(ra::SeqProb* P, int n_seqs, int Hq, int Hkv, int total_q, int dtype, double scale) {
  memset(P, 0, sizeof(*P));
  P->n_seqs = n_seqs;
  P->Hq = Hq;
  P->Hkv = Hkv;
  P->G = Hq / Hkv;
  P->inv_G = (65536 + P->G - 1) / P->G;
  P->TQ = 128 / P->G;
  P->total_q = total_q;
  P->bf16 = dtype == RA_BF16;
  P->cs = log2_scale(scale);
}

bool q_map(ra::SeqMaps* m, const ra::SeqProb& P, const void* q, long long tok, long long head) {
  const cuuint64_t outer[3] = {(cuuint64_t)P.G, (cuuint64_t)P.Hkv, (cuuint64_t)P.total_q};
  const cuuint64_t h = map_stride(head, P.Hq);
  const cuuint64_t stride[3] = {h, h * P.G, map_stride(tok, P.total_q)};
  const cuuint32_t box[3] = {(cuuint32_t)P.G, 1, (cuuint32_t)P.TQ};
  return make_map(&m->q, P.bf16, q, outer, stride, box);
}

void bind_ws(ra::SeqProb* P, int many, int few, void* ws) {
  const ra::SeqWs L = ra::seq_ws(P->n_seqs, P->total_q, P->Hq, P->shared, many, few);
  char* b = static_cast<char*>(ws);
  P->err = &static_cast<ra::WsHeader*>(ws)->err;
  auto floats = [&](size_t o) { return reinterpret_cast<float*>(b + o); };
  P->many.starts = reinterpret_cast<long long*>(b + L.many_starts);
  P->many.split = reinterpret_cast<ra::SplitItem*>(b + L.many_split);
  P->few.split = reinterpret_cast<ra::SplitItem*>(b + L.few_split);
  P->many.slot_o = floats(L.many_o);
  P->many.slot_lse = floats(L.many_lse);
  P->few.starts = reinterpret_cast<long long*>(b + L.few_starts);
  P->few.slot_o = floats(L.few_o);
  P->few.slot_lse = floats(L.few_lse);
  P->lead_o = floats(L.lead_o);
  P->lead_lse = floats(L.lead_lse);
  P->own_o = floats(L.own_o);
  P->own_lse = floats(L.own_lse);
}

// Which kernels a cache call may need: sequences of unknown query lengths may
// go to either.
void cache_kinds(const ra_cache_attn* a, int G, bool single, bool* many, bool* few) {
  const bool lead_few = (long long)a->total_q * G <= ra::FEW_ROWS, one_few = G <= ra::FEW_ROWS;
  *few = one_few;
  *many = (a->shared > 0 && !lead_few) || (single ? !one_few : !lead_few);
}

}  // namespace

extern "C" {

size_t ra_packed_workspace_bytes(const ra_packed* p) {
  if (check_packed(p) != RA_OK) return 0;
  if (!packed_split(p)) return align256(sizeof(ra::WsHeader));
  return ra::seq_ws(p->n_seqs, p->total_q, p->Hq, 0, SM_BOUND, 0).total;
}

ra_status ra_packed_attention_fwd(const ra_packed* p, const void* q, const void* k, const void* v, const int* cu_q,
                                  const int* cu_k, void* o, float* lse, void* ws, size_t ws_bytes, ra_stream stream) {
  ra_status st = check_packed(p);
  if (st != RA_OK) return st;
  if (!aligned(ws, 256)) return fail(RA_ERR_INVALID_ARG, "workspace pointer NULL or not 256-byte aligned");
  const size_t need = ra_packed_workspace_bytes(p);
  if (ws_bytes < need) return fail(RA_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, need);
  if (!aligned(cu_q, 4) || !aligned(cu_k, 4)) return fail(RA_ERR_INVALID_ARG, "cu_q or cu_k NULL or misaligned");
  if (p->total_q == 0) return RA_OK;
  if (!aligned(q, 16) || !aligned(o, 16)) return fail(RA_ERR_INVALID_ARG, "q or o NULL or not 16-byte aligned");
  if (p->total_k > 0 && (!aligned(k, 16) || !aligned(v, 16)))
    return fail(RA_ERR_INVALID_ARG, "k or v NULL or not 16-byte aligned");
  if (lse != nullptr && !aligned(lse, 4)) return fail(RA_ERR_INVALID_ARG, "lse misaligned");
  ra::SeqProb P;
  fill_common(&P, p->n_seqs, p->Hq, p->Hkv, p->total_q, p->dtype, p->scale);
  P.total_k = p->total_k;
  P.causal = p->causal;
  P.cu_q = cu_q;
  P.cu_k = cu_k;
  P.page_shift = 7;
  P.page_size = 128;
  P.v = static_cast<const uint8_t*>(v);
  P.v_tok = 2 * p->v_token;
  P.v_head = 2 * p->v_head;
  P.o = static_cast<uint8_t*>(o);
  P.o_tok = 2 * p->o_token;
  P.o_head = 2 * p->o_head;
  P.lse = lse;
  P.items = packed_items(p->total_q, p->n_seqs, P.TQ, P.Hkv);
  P.split = packed_split(p);
  int sms = 0;
  if ((st = sm_count(&sms)) != RA_OK) return st;
  P.many.grid = sms < SM_BOUND ? sms : SM_BOUND;
  if (!P.split && P.items < P.many.grid) P.many.grid = (int)P.items;
  if (P.split) bind_ws(&P, SM_BOUND, 0, ws);
  ra::SeqMaps m;
  const void* kb = p->total_k > 0 ? k : q;   // no keys at all: no copy of them is issued
  const void* vb = p->total_k > 0 ? v : q;
  const cuuint64_t rows = p->total_k > 0 ? p->total_k : 1;
  const cuuint64_t outer[3] = {1, (cuuint64_t)p->Hkv, rows};
  const cuuint64_t ks[3] = {256, map_stride(p->k_head, p->Hkv), map_stride(p->k_token, p->total_k)};
  const cuuint64_t vs[3] = {256, map_stride(p->v_head, p->Hkv), map_stride(p->v_token, p->total_k)};
  const cuuint32_t box[3] = {1, 1, ra::KEYS};
  if (!q_map(&m, P, q, p->q_token, p->q_head) || !make_map(&m.k, P.bf16, kb, outer, ks, box) ||
      !make_map(&m.v, P.bf16, vb, outer, vs, box))
    return fail(RA_ERR_CUDA, "tensor map of q, k or v");
  const cudaError_t e = ra::launch_seq_attention(P, m, ws, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? RA_OK : cuda_fail(e, "packed attention launch");
}

ra_status ra_cache_validate(const ra_cache_problem* p) { return check_cache(p, nullptr); }

size_t ra_cache_pool_bytes(const ra_cache_problem* p) {
  return check_cache(p, nullptr) == RA_OK ? 2 * half_pool(p) : 0;
}

size_t ra_cache_state_bytes(const ra_cache_problem* p) {
  if (check_cache(p, nullptr) != RA_OK) return 0;
  return align256(4 * (size_t)p->n_pages) + align256(4 * (size_t)p->max_seqs) +
         align256(4 * (size_t)p->max_seqs * p->max_pages);
}

ra_status ra_cache_bind(const ra_cache_problem* p, void* pool, size_t pool_bytes, void* state, size_t state_bytes,
                        ra_cache* out) {
  const ra_status st = check_cache(p, nullptr);
  if (st != RA_OK) return st;
  if (out == nullptr) return fail(RA_ERR_INVALID_ARG, "output ra_cache is NULL");
  if (!aligned(pool, 256) || !aligned(state, 256))
    return fail(RA_ERR_INVALID_ARG, "pool or state NULL or not 256-byte aligned");
  if (pool_bytes < ra_cache_pool_bytes(p) || state_bytes < ra_cache_state_bytes(p))
    return fail(RA_ERR_INVALID_ARG, "pool or state smaller than %zu and %zu bytes", ra_cache_pool_bytes(p),
                ra_cache_state_bytes(p));
  char* s = static_cast<char*>(state);
  out->k = pool;
  out->v = static_cast<char*>(pool) + half_pool(p);
  out->refs = reinterpret_cast<int*>(s);
  s += align256(4 * (size_t)p->n_pages);
  out->lens = reinterpret_cast<int*>(s);
  s += align256(4 * (size_t)p->max_seqs);
  out->table = reinterpret_cast<int*>(s);
  return RA_OK;
}

size_t ra_cache_workspace_bytes(const ra_cache_problem* p) {
  return check_cache(p, nullptr) == RA_OK ? ra::cache_ws(p->n_pages, p->max_seqs).total : 0;
}

ra_status ra_cache_init(const ra_cache_problem* p, const ra_cache* c, ra_stream stream) {
  const ra_status st = check_cache(p, nullptr);
  if (st != RA_OK) return st;
  if (c == nullptr || !aligned(c->refs, 16) || !aligned(c->lens, 16) || !aligned(c->table, 16))
    return fail(RA_ERR_INVALID_ARG, "a cache pointer is NULL or not 16-byte aligned");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaMemsetAsync(c->refs, 0, 4 * (size_t)p->n_pages, s);
  if (e == cudaSuccess) e = cudaMemsetAsync(c->lens, 0, 4 * (size_t)p->max_seqs, s);
  if (e == cudaSuccess) e = cudaMemsetAsync(c->table, 0xFF, 4 * (size_t)p->max_seqs * p->max_pages, s);
  return e == cudaSuccess ? RA_OK : cuda_fail(e, "cache init");
}

ra_status ra_cache_extend(const ra_cache_problem* p, const ra_cache* c, const int* seqs, const int* n_new, int n,
                          void* ws, size_t ws_bytes, ra_stream stream) {
  ra::CacheProb C;
  ra_status st = check_cache_call(p, c, ws, ws_bytes, &C);
  if (st != RA_OK || (st = check_list(seqs, n, p->max_seqs)) != RA_OK || (st = check_list(n_new, n, p->max_seqs)) != RA_OK)
    return st;
  if (n == 0) return RA_OK;
  const cudaError_t e = ra::launch_cache_extend(C, seqs, n_new, n, ws, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? RA_OK : cuda_fail(e, "cache extend launch");
}

ra_status ra_cache_write(const ra_cache_problem* p, const ra_cache* c, int layer, const int* seqs, const int* cu_new,
                         int n, int total, const void* k, const void* v, long long k_token, long long k_head,
                         long long v_token, long long v_head, void* ws, size_t ws_bytes, ra_stream stream) {
  ra::CacheProb C;
  ra_status st = check_cache_call(p, c, ws, ws_bytes, &C);
  if (st != RA_OK || (st = check_list(seqs, n, p->max_seqs)) != RA_OK) return st;
  if (layer < 0 || layer >= p->layers) return fail(RA_ERR_INVALID_ARG, "layer %d of %d", layer, p->layers);
  if (total < 0 || (cu_new == nullptr && total != n) || (n == 0 && total > 0))
    return fail(RA_ERR_INVALID_ARG, "%d tokens for %d rows", total, n);
  if (cu_new != nullptr && !aligned(cu_new, 4)) return fail(RA_ERR_INVALID_ARG, "cu_new misaligned");
  if (n == 0) return RA_OK;
  if (total > (1 << 24)) return fail(RA_ERR_UNSUPPORTED, "at most 2^24 tokens per call");
  if (total > 0 && (!aligned(k, 16) || !aligned(v, 16))) return fail(RA_ERR_INVALID_ARG, "k or v NULL or not 16-byte aligned");
  if ((st = check_strides("k", k_token, k_head, total, p->Hkv)) != RA_OK) return st;
  if ((st = check_strides("v", v_token, v_head, total, p->Hkv)) != RA_OK) return st;
  if ((long long)total * p->Hkv >= (1ll << 33)) return fail(RA_ERR_UNSUPPORTED, "too many rows for one call");
  const cudaError_t e = ra::launch_cache_write(C, layer, seqs, cu_new, n, total, static_cast<const uint8_t*>(k),
                                               static_cast<const uint8_t*>(v), 2 * k_token, 2 * k_head, 2 * v_token,
                                               2 * v_head, ws, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? RA_OK : cuda_fail(e, "cache write launch");
}

ra_status ra_cache_fork(const ra_cache_problem* p, const ra_cache* c, const int* parents, const int* children, int n,
                        void* ws, size_t ws_bytes, ra_stream stream) {
  ra::CacheProb C;
  ra_status st = check_cache_call(p, c, ws, ws_bytes, &C);
  if (st != RA_OK || (st = check_list(parents, n, p->max_seqs)) != RA_OK ||
      (st = check_list(children, n, p->max_seqs)) != RA_OK)
    return st;
  if (n == 0) return RA_OK;
  const cudaError_t e = ra::launch_cache_fork(C, parents, children, n, ws, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? RA_OK : cuda_fail(e, "cache fork launch");
}

ra_status ra_cache_free(const ra_cache_problem* p, const ra_cache* c, const int* seqs, int n, void* ws,
                        size_t ws_bytes, ra_stream stream) {
  ra::CacheProb C;
  ra_status st = check_cache_call(p, c, ws, ws_bytes, &C);
  if (st != RA_OK || (st = check_list(seqs, n, p->max_seqs)) != RA_OK) return st;
  if (n == 0) return RA_OK;
  const cudaError_t e = ra::launch_cache_free(C, seqs, n, ws, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? RA_OK : cuda_fail(e, "cache free launch");
}

ra_status ra_cache_compact(const ra_cache_problem* p, const ra_cache* c, void* ws, size_t ws_bytes, ra_stream stream) {
  ra::CacheProb C;
  const ra_status st = check_cache_call(p, c, ws, ws_bytes, &C);
  if (st != RA_OK) return st;
  const cudaError_t e = ra::launch_cache_compact(C, ws, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? RA_OK : cuda_fail(e, "cache compact launch");
}

size_t ra_cache_attention_workspace_bytes(const ra_cache_problem* p, const ra_cache_attn* a) {
  if (check_attn(p, a) != RA_OK) return 0;
  bool many, few;   // with cu_q, which needs the most
  cache_kinds(a, a->Hq / p->Hkv, false, &many, &few);
  return ra::seq_ws(a->n_seqs, a->total_q, a->Hq, a->shared, many ? SM_BOUND : 0, few ? ra::FEW_CTAS * SM_BOUND : 0).total;
}

ra_status ra_cache_attention_fwd(const ra_cache_problem* p, const ra_cache* c, const ra_cache_attn* a, const void* q,
                                 const int* seqs, const int* cu_q, void* o, float* lse, void* ws, size_t ws_bytes,
                                 ra_stream stream) {
  ra_status st = check_attn(p, a);
  if (st != RA_OK) return st;
  if (c == nullptr || !aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->lens, 16) || !aligned(c->table, 16))
    return fail(RA_ERR_INVALID_ARG, "a cache pointer is NULL or not 16-byte aligned");
  if (!aligned(ws, 256)) return fail(RA_ERR_INVALID_ARG, "workspace pointer NULL or not 256-byte aligned");
  const size_t need = ra_cache_attention_workspace_bytes(p, a);
  if (ws_bytes < need) return fail(RA_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, need);
  if (!aligned(seqs, 4) || (cu_q != nullptr && !aligned(cu_q, 4)))
    return fail(RA_ERR_INVALID_ARG, "seqs NULL, or seqs or cu_q misaligned");
  if (cu_q == nullptr && a->total_q != a->n_seqs)
    return fail(RA_ERR_INVALID_ARG, "%d query rows for %d single tokens", a->total_q, a->n_seqs);
  if (a->total_q == 0) return RA_OK;
  if (!aligned(q, 16) || !aligned(o, 16)) return fail(RA_ERR_INVALID_ARG, "q or o NULL or not 16-byte aligned");
  if (lse != nullptr && !aligned(lse, 4)) return fail(RA_ERR_INVALID_ARG, "lse misaligned");
  ra::CacheProb C;
  check_cache(p, &C);
  ra::SeqProb P;
  fill_common(&P, a->n_seqs, a->Hq, p->Hkv, a->total_q, p->dtype, a->scale);
  P.causal = 1;
  P.cu_q = cu_q;
  P.paged = 1;
  P.shared = a->shared;
  P.page_size = C.page_size;
  P.page_shift = C.page_shift;
  P.max_pages = C.max_pages;
  P.n_pages = C.n_pages;
  P.max_seqs = C.max_seqs;
  P.seqs = seqs;
  P.lens = c->lens;
  P.table = c->table;
  const size_t layer = (size_t)256 * p->n_pages * p->Hkv * p->page_size;
  const uint8_t* kb = static_cast<const uint8_t*>(c->k) + a->layer * layer;
  const uint8_t* vb = static_cast<const uint8_t*>(c->v) + a->layer * layer;
  P.q = static_cast<const uint8_t*>(q);
  P.q_tok = 2 * a->q_token;
  P.q_head = 2 * a->q_head;
  P.k = kb;
  P.v = vb;
  P.v_tok = 256;
  P.v_head = 256ll * p->page_size;
  P.v_page = P.v_head * p->Hkv;
  P.o = static_cast<uint8_t*>(o);
  P.o_tok = 2 * a->o_token;
  P.o_head = 2 * a->o_head;
  P.lse = lse;
  P.split = 1;
  int sms = 0;
  if ((st = sm_count(&sms)) != RA_OK) return st;
  if (sms > SM_BOUND) sms = SM_BOUND;
  bool many, few;
  cache_kinds(a, P.G, false, &many, &few);
  bind_ws(&P, many ? SM_BOUND : 0, few ? ra::FEW_CTAS * SM_BOUND : 0, ws);
  cache_kinds(a, P.G, cu_q == nullptr, &many, &few);
  // one head per warp while that fits the SMs at once; more per lookup else
  P.join_heads = (long long)a->total_q * a->Hq <= 64ll * SM_BOUND ? 8 : 32;
  P.lead_only = cu_q == nullptr && P.G <= ra::FEW_ROWS;
  // A short shared region, of at most LEAD_TILES key tiles per SM on half of
  // them, leaves the others to the kernel of few rows, which runs beside it (the
  // host does not know the own lengths, but with half of the SMs they take at most
  // twice their time); a longer one gets the whole GPU, and so does the kernel of
  // few rows behind it.  Beside / one after the other: own lengths 1 to 1024 of 61
  // rows, 32/8 heads, 2048 shared tokens (43 SMs) 31 / 44 us, 2944 (62 SMs) 35 /
  // 45; 5683 to 15646 of 25 rows, 40/8 heads, 237 / 202 and 285 / 210.  (Beside a
  // region on all SMs but one they take 22 ms.)
  constexpr long long LEAD_TILES = 3;
  P.many.grid = many ? sms : 0;
  if (many && P.lead_only) {
    const long long tiles = (long long)((a->shared + ra::KEYS - 1) / ra::KEYS) * p->Hkv *
                            ((a->total_q + 2 * P.TQ - 1) / (2 * P.TQ));
    const long long want = (tiles + LEAD_TILES - 1) / LEAD_TILES;
    if (want <= sms / 2) P.many.grid = (int)want;
  }
  P.few.grid = few ? ra::FEW_CTAS * (P.many.grid < sms ? sms - P.many.grid : sms) : 0;
  ra::SeqMaps m;
  const cuuint64_t outer[3] = {(cuuint64_t)p->page_size, (cuuint64_t)p->Hkv, (cuuint64_t)p->n_pages};
  const cuuint64_t stride[3] = {256, (cuuint64_t)P.v_head, (cuuint64_t)P.v_page};
  const cuuint32_t box[3] = {(cuuint32_t)p->page_size, 1, 1};
  if (many && (!q_map(&m, P, q, a->q_token, a->q_head) || !make_map(&m.k, P.bf16, kb, outer, stride, box) ||
               !make_map(&m.v, P.bf16, vb, outer, stride, box)))
    return fail(RA_ERR_CUDA, "tensor map of q or the pool");
  const cudaError_t e = ra::launch_seq_attention(P, m, ws, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? RA_OK : cuda_fail(e, "cache attention launch");
}

}  // extern "C"
