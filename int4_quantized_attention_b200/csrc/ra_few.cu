// ra_few.cu -- attention of at most 64 query rows (a token, or a few, of one
// sequence, with the query heads that share a key head) over the pages of a
// cache: the decoding step.
//
// Mathematics: as ra_packed.cu, o = sum_j p_j v_j / sum_j p_j.  Each K and V
// element is used by 1 to 64 rows only, so the pages' bytes set the pace (512
// bytes per token and key head), not the products.  Hence
//   - three small CTAs per SM rather than one large pipeline: what one waits
//     for (page numbers, the join of its warps, the first tile of its next
//     item), the others hide;
//   - the warp-level MMA (m16n8k16): 16 rows cost 32 of them per 16 keys, where
//     a tensor-memory tile would be 128 rows high and its softmax would have
//     to go through them;
//   - K and V tiles of 64 keys by 16-byte asynchronous copies, which fetch any
//     page layout at the same cost and fill slots past the region's end with
//     zeros, so that what lies there (NaN, say) never reaches a product.
//
// A CTA's four warps share the tile's keys: with R 16-row blocks of queries (R
// = 1, 2, 4), warp w works for block w % R on keys 16 R (w / R) .. + 16 R - 1,
// 16 at a time, with a running maximum, sum and fp32 accumulator of its own; the
// 4 / R partial results of each row are joined through shared memory at the
// end of the part.  The work is dealt as in the split form of ra_packed.cu:
// equal shares of all keys, parts of an item put together by the joining kernel.
//
// What it measured: 24 sequences of 8000 tokens, 40/8 heads (787 MB): 126 us,
// 6.22 TB/s, 0.95 of the measured copy.  On the 128-row tiles the same call took
// 160 us, and 48 sequences of 1 to 16384 tokens 228 us where it takes 90: short
// parts cost a pipeline of one CTA per SM its full latency each time.  A part
// costs some 9,000 cycles besides its tiles (3,800 each, three CTAs sharing the
// memory), which W_ITEM charges it for.
#include "ra_seq.cuh"

namespace ra {
namespace {

constexpr int THREADS = 128;
constexpr uint32_t HALF_STAGE = FEW_KEYS * 256;       // K or V of a tile: 16 KB
constexpr uint32_t RING = 2 * 2 * HALF_STAGE;         // two stages; afterwards the warps' rows, 4 x 16 x 512 bytes
constexpr int NO_COPY = 0x1ffffff;                    // a tile past every region's end
static_assert(RING >= 4 * 16 * D * sizeof(float), "join space");

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
template <int N>
__device__ __forceinline__ void wait_copies() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
template <bool BF16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 16-byte piece c (of 16) of 256-byte row r of a tile: the low three bits of
// the piece are XORed with the row, so that eight rows of one piece lie in
// eight different places of the 128-byte bank line.
__device__ __forceinline__ uint32_t tile_off(uint32_t r, uint32_t c) { return r * 256u + ((c ^ (r & 7u)) << 4); }

template <bool BF16>
__global__ void __launch_bounds__(THREADS, FEW_CTAS) few_kernel(const __grid_constant__ SeqProb P, WsHeader* __restrict__ hdr) {
  constexpr float BIAS = BF16 ? 0.0f : 7.0f;   // fp16 weights carry a factor 2^7
  extern __shared__ __align__(1024) uint8_t sm[];
  __shared__ SharePlan plan;
  __shared__ float stat_m[4][16], stat_l[4][16];   // per warp and row of its block
  __shared__ int nf_tile;                           // first tile with values taken out of V
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  DeviceErr* err = &hdr->err;
  dependents_may_start();
  plan_shares<KIND_FEW, THREADS>(P, plan, err);
  ShareWalk<KIND_FEW> w;
  start_walk(P, plan, w);
  SplitItem* const split = P.few.split + blockIdx.x;
  if (tid == 0) split->parts = 0;
  const uint32_t ring = smem_u32(sm);
  const int copy_row = tid >> 4, copy_piece = tid & 15;   // this thread's rows of a tile: copy_row + 8 i
  SharePart part;
  while (next_share_part(P, plan, w, part, err)) {
    const int rows = part.tokens * P.G, n = part.t1 - part.t0;
    const int blocks = rows <= 16 ? 1 : rows <= 32 ? 2 : 4, groups = 4 / blocks;
    const int block = warp & (blocks - 1), group = warp >> (blocks >> 1);
    const int q0 = part.lead ? 0 : w.s.q0, table_row = part.lead ? plan.lead_row : w.s.row;
    const int key0 = part.lead ? 0 : P.shared, off = part.lead ? 0 : w.s.off;
    const int len = part.lead ? min(P.shared, plan.lead_len) : w.s.len;
    const long long head_off = (long long)part.kvh * P.v_head;
    const int* pages = P.table + (long long)table_row * P.max_pages;
    // K and V of tile t (of the region), this thread's 2 x 8 pieces
    auto copy_tile = [&](int t, int stage) {
      const uint32_t k_dst = ring + stage * 2 * HALF_STAGE, v_dst = k_dst + HALF_STAGE;
      int page = -1, slot = -1;
      // past the part's end nothing is copied: not even zeros, which would land
      // on the rows that faster warps already lay out for the join
#pragma unroll
      for (int i = 0; i < FEW_KEYS / 8; ++i) {
        if (t == NO_COPY) break;
        const int r = copy_row + 8 * i, key = t * FEW_KEYS + r, pos = key0 + key;
        bool there = key < len;
        if (there && (pos >> P.page_shift) != slot) {
          slot = pos >> P.page_shift;
          page = __ldg(pages + slot);
          if ((uint32_t)page >= (uint32_t)P.n_pages) {   // not a page: read as zeros
            report(err, DEVERR_BOUNDS, 0x4501);
            page = -1;
          }
        }
        there = there && page >= 0 &&
                in_bounds(slot < P.max_pages && table_row < P.max_seqs && part.kvh < P.Hkv &&
                              head_off + (pos & (P.page_size - 1)) * 256 + 256 <= P.v_page, err, 0x4504);
        const long long at = there ? page * P.v_page + head_off + (pos & (P.page_size - 1)) * 256 + copy_piece * 16 : 0;
        copy16(k_dst + tile_off(r, copy_piece), P.k + at, there);
        copy16(v_dst + tile_off(r, copy_piece), P.v + at, there);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if (tid == 0) nf_tile = NO_TILE;
    if (tid == 0 && part.out == OUT_SLOT && (part.slot & 1)) *split = {part.parts, q0, part.tokens, part.kvh};
    // this warp's 16 rows of Q as operand registers; rows past the last are zero
    uint32_t q[8][4];
    int lim[2], gmin = len;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = 16 * block + 8 * i + (lane >> 2), t = over_G(P, min(r, rows - 1));
      const bool real = r < rows;
      const uint8_t* src = P.q + (q0 + t) * P.q_tok + (part.kvh * P.G + min(r, rows - 1) - t * P.G) * P.q_head + 4 * (lane & 3);
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        q[kk][i] = real ? *reinterpret_cast<const uint32_t*>(src + 32 * kk) : 0u;
        q[kk][2 + i] = real ? *reinterpret_cast<const uint32_t*>(src + 32 * kk + 16) : 0u;
      }
      lim[i] = real ? row_limit(P, part.lead, off, len, t) : 0;
    }
    // keys that every row sees: the first row's, or the least of all of them
    if (part.lead) {
      for (int t = lane; t < part.tokens; t += 32) gmin = min(gmin, lead_limit(P, len, t));
      gmin = __reduce_min_sync(0xffffffffu, gmin);
    } else {
      gmin = row_limit(P, 0, off, len, 0);
    }
    float o[16][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < 16; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[c][e] = 0.0f;

    // tiles are copied two ahead; the body stands once, for the instruction cache
#pragma unroll 1
    for (int t = -2; t < n; ++t) {
      const int key = (part.t0 + t) * FEW_KEYS, stage = t & 1;
      if (t >= 0) {
      wait_copies<1>();
      __syncthreads();
      const uint32_t kt = ring + stage * 2 * HALF_STAGE, vt = kt + HALF_STAGE;
      if (key + FEW_KEYS > gmin && gmin < len) {
        // values that some row must not see meet a zero weight there, and 0 x
        // infinity is NaN: non-finite ones become zero here, and are added
        // back at the end for the rows that see them
        for (int c = tid; c < FEW_KEYS * 16; c += THREADS) {
          const int r = c >> 4;
          if (key + r < gmin) continue;
          uint4* at = reinterpret_cast<uint4*>(sm + (vt - ring) + tile_off(r, c & 15));
          uint4 v = *at;
          uint32_t* x = reinterpret_cast<uint32_t*>(&v);
          bool bad = false;
          for (int e = 0; e < 4; ++e) {
            if (nonfinite16<BF16>(x[e])) x[e] &= 0xffff0000u, bad = true;
            if (nonfinite16<BF16>(x[e] >> 16)) x[e] &= 0xffffu, bad = true;
          }
          if (bad) {
            *at = v;
            atomicMin(&nf_tile, part.t0 + t);
          }
        }
        __syncthreads();
      }
#pragma unroll 1
      for (int b = 0; b < blocks; ++b) {
        const int k16 = 16 * (group * blocks + b);   // 16 keys of the tile
        float s[2][4] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
        const uint32_t k_row = k16 + (lane & 7) + ((lane >> 4) & 1) * 8;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          uint32_t kf[4];
          ldmatrix4(kf, kt + tile_off(k_row, 2 * kk + ((lane >> 3) & 1)));
          mma16816<BF16>(s[0], q[kk], kf[0], kf[1]);
          mma16816<BF16>(s[1], q[kk], kf[2], kf[3]);
        }
        uint32_t p[4];
        float alpha[2];
        bool moved[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float x[4] = {s[0][2 * i], s[0][2 * i + 1], s[1][2 * i], s[1][2 * i + 1]};
          if (key + FEW_KEYS > gmin) {
            const int first = key + k16 + 2 * (lane & 3);
            if (first >= lim[i]) x[0] = -INFINITY;
            if (first + 1 >= lim[i]) x[1] = -INFINITY;
            if (first + 8 >= lim[i]) x[2] = -INFINITY;
            if (first + 9 >= lim[i]) x[3] = -INFINITY;
          }
          float mx = max3_nan(max3_nan(x[0], x[1], x[2]), x[3], x[3]);
          float y = __shfl_xor_sync(0xffffffffu, mx, 1);
          mx = max3_nan(mx, y, y);
          y = __shfl_xor_sync(0xffffffffu, mx, 2);
          mx = max3_nan(mx, y, y) * P.cs;
          moved[i] = !(mx <= m[i] + RAISE);
          const float m_new = moved[i] ? (mx == INFINITY ? NAN : mx) : m[i];
          alpha[i] = moved[i] ? ex2(m[i] - m_new) : 1.0f;
          m[i] = m_new;
          const float add = BIAS - (m_new == -INFINITY ? 0.0f : m_new);
          const float p0 = ex2(fmaf(x[0], P.cs, add)), p1 = ex2(fmaf(x[1], P.cs, add));
          const float p2 = ex2(fmaf(x[2], P.cs, add)), p3 = ex2(fmaf(x[3], P.cs, add));
          l[i] = fmaf(l[i], alpha[i], (p0 + p1) + (p2 + p3));
          p[i] = pack2<BF16>(p0, p1);
          p[2 + i] = pack2<BF16>(p2, p3);
        }
        if (__any_sync(0xffffffffu, moved[0] || moved[1])) {
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            o[c][0] *= alpha[0];
            o[c][1] *= alpha[0];
            o[c][2] *= alpha[1];
            o[c][3] *= alpha[1];
          }
        }
        const uint32_t v_row_ = k16 + (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          uint32_t vf[4];
          ldmatrix4_trans(vf, vt + tile_off(v_row_, 2 * c + (lane >> 4)));
          mma16816<BF16>(o[2 * c], p, vf[0], vf[1]);
          mma16816<BF16>(o[2 * c + 1], p, vf[2], vf[3]);
        }
      }
      __syncthreads();   // the stage has been read
      }
      copy_tile(t + 2 < n ? part.t0 + t + 2 : NO_COPY, stage);
    }
    wait_copies<0>();

    // join the groups' rows
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float x = l[i];
      x += __shfl_xor_sync(0xffffffffu, x, 1);
      x += __shfl_xor_sync(0xffffffffu, x, 2);
      if ((lane & 3) == 0) {
        stat_m[warp][8 * i + (lane >> 2)] = m[i];
        stat_l[warp][8 * i + (lane >> 2)] = x;
      }
    }
    float* join = reinterpret_cast<float*>(sm);   // [warp][16 rows][128], 16-byte pieces XORed with the row
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      const int r = lane >> 2, piece = (2 * c + ((lane >> 1) & 1)) ^ r;
      float* d = join + (warp * 16 + r) * D + 4 * piece + 2 * (lane & 1);
      *reinterpret_cast<float2*>(d) = make_float2(o[c][0], o[c][1]);
      *reinterpret_cast<float2*>(d + 8 * D) = make_float2(o[c][2], o[c][3]);
    }
    __syncthreads();
    const int nf = nf_tile;
    // a row's factors, once: 2^(m - M) / L of each group
    if (tid < rows) {
      const int b = tid >> 4, r = tid & 15;
      float M = -INFINITY, L = 0.0f;
      for (int g = 0; g < groups; ++g) M = max3_nan(M, stat_m[g * blocks + b][r], M);
      for (int g = 0; g < groups; ++g) {
        const int v = g * blocks + b;
        const float f = stat_m[v][r] == -INFINITY ? 0.0f : ex2(stat_m[v][r] - M);
        L = fmaf(f, stat_l[v][r], L);
        stat_m[v][r] = f;
      }
      const float inv = L != 0.0f ? 1.0f / L : 0.0f;   // a row without keys: zeros
      for (int g = 0; g < groups; ++g) stat_m[g * blocks + b][r] *= inv;
      const int t = over_G(P, tid), token = q0 + t, head = part.kvh * P.G + tid - t * P.G;
      const RowOut out = row_out(P, P.few, part.out, part.slot, token, head, tid, FEW_ROWS);
      const float lse2 = L != 0.0f ? M - BIAS + log2f(L) : -INFINITY;
      if (out.lse != nullptr && in_bounds(row_inside(P, P.few, part.out, part.slot, token, head, tid, FEW_ROWS), err, 0x4503))
        *out.lse = part.out == OUT_FINAL ? lse2 * LN2 : lse2;
    }
    __syncthreads();
#pragma unroll 2
    for (int row = tid >> 4; row < rows; row += 8) {
      const int c8 = (tid & 15) * 8, b = row >> 4, r = row & 15;
      float y[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        if (g >= groups) continue;
        const int v = g * blocks + b;
        const float f = stat_m[v][r];
        const float4* x = reinterpret_cast<const float4*>(join + (v * 16 + r) * D);
        const float4 x0 = x[(c8 / 4) ^ (r & 7)], x1 = x[(c8 / 4 + 1) ^ (r & 7)];
        y[0] = fmaf(f, x0.x, y[0]);
        y[1] = fmaf(f, x0.y, y[1]);
        y[2] = fmaf(f, x0.z, y[2]);
        y[3] = fmaf(f, x0.w, y[3]);
        y[4] = fmaf(f, x1.x, y[4]);
        y[5] = fmaf(f, x1.y, y[5]);
        y[6] = fmaf(f, x1.z, y[6]);
        y[7] = fmaf(f, x1.w, y[7]);
      }
      const int t = over_G(P, row), token = q0 + t, head = part.kvh * P.G + row - t * P.G;
      if (nf != NO_TILE) {
        float z[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] = y[e];
        add_nonfinite<BF16, 8>(P, {key0, table_row, part.kvh}, nf * FEW_KEYS,
                               min(row_limit(P, part.lead, off, len, t), part.t1 * FEW_KEYS), c8, z);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = z[e];
      }
      if (in_bounds(row_inside(P, P.few, part.out, part.slot, token, head, row, FEW_ROWS), err, 0x4502))
        store8<BF16>(row_out(P, P.few, part.out, part.slot, token, head, row, FEW_ROWS), c8, y);
    }
    __syncthreads();   // the ring is free for the next part
  }
  // the kernel of many rows may still run: this grid ends after it, so that
  // the join, which waits for this one, finds both results
  wait_for_predecessor();
}

template <bool BF16>
cudaError_t launch(const SeqProb& p, WsHeader* hdr, bool overlap, cudaStream_t st) {
  static OncePerDevice once;
  const cudaError_t e = once.run(
      [] { return cudaFuncSetAttribute(few_kernel<BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, RING); });
  if (e != cudaSuccess) return e;
  return launch_after(overlap, few_kernel<BF16>, p.few.grid, THREADS, RING, st, p, hdr);
}

}  // namespace

cudaError_t launch_few_attention(const SeqProb& p, WsHeader* hdr, bool overlap, cudaStream_t st) {
  return p.bf16 ? launch<true>(p, hdr, overlap, st) : launch<false>(p, hdr, overlap, st);
}

}  // namespace ra
