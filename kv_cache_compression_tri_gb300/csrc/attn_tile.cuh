// attn_tile.cuh -- the CUDA-core forms (fp32 caches) of attention over a chunk of
// queries: tiles of 64 packed query rows (tokens x the group's heads) by 64 cached rows
// in fp32 shared memory, 4 x 4 logits per thread.
#pragma once

#include "attn_common.cuh"

namespace tri {
namespace {

constexpr int FT = 256;  // threads per CTA
constexpr int FM = 64;   // packed query rows of a tile
constexpr int FN = 64;   // cached rows of a tile

// A chunk's place in the cache: one (sequence, KV head).
struct Chunk {
  int64_t s;       // slice of the cache
  int n, seq, h;   // valid rows, sequence, KV head
  int n_new, r0;   // new tokens; row of token 0's query (may be negative)
};

// false: nothing to do for this sequence, or a fault (reported).
__device__ __forceinline__ bool chunk_of(const AttnParams& p, int ls, Chunk& c) {
  c.seq = ls / p.n_kv_heads;
  c.h = ls - c.seq * p.n_kv_heads;
  c.s = slice_of(p, c.seq, c.h);
  c.n = p.n_valid[c.s];
  c.n_new = new_tokens(p, c.seq);
  c.r0 = c.n - c.n_new;
  if (c.n < 0 || c.n > p.n_cap) {
    set_status(p.dev_status, TRI_DEV_NVALID_OVER_CAP);
    return false;
  }
  return c.n_new > 0;
}

// Whether any query of rows r_first .. r_last sees a row of [k0, k0 + len)
// (r_first may be negative: the first query that sees anything is at row 0 then).
__device__ __forceinline__ bool tile_seen(const AttnParams& p, int k0, int len, int r_first, int r_last) {
  if (k0 > r_last) return false;
  return p.window == 0 || k0 < p.n_sink || k0 + len - 1 > max(r_first, 0) - p.window;
}

__device__ __forceinline__ bool sees(const AttnParams& p, int r, int j) {
  return j <= r && (p.window == 0 || j < p.n_sink || j > r - p.window);
}

// The table entries of every row that rows r_first .. r_last see are in the
// pool (by the CTA; the slice is skipped and reported otherwise).
__device__ __forceinline__ bool chunk_blocks_ok(const AttnParams& p, const int32_t* trow, int r_first, int r_last, int* flag) {
  const Visible first = visible_rows(max(r_first, 0), p.n_sink, p.window);
  const Visible last = visible_rows(max(r_last, 0), p.n_sink, p.window);
  bool ok = p.rows.blocks_ok(trow, 0, last.s1, flag);
  ok = p.rows.blocks_ok(trow, first.w0, r_last + 1, flag) && ok;
  if (!ok && threadIdx.x == 0) set_status(p.dev_status, TRI_DEV_BAD_BLOCK);
  return ok;
}

// Packed rows [0, FM) of queries: row u is token tok0 + u / group, head u % group.
template <int D>
__device__ __forceinline__ void load_queries(const AttnParams& p, const Chunk& c, int tok0, int rows, float (*sq)[D + 4]) {
  constexpr int C = D / 4;
  for (int i = threadIdx.x; i < FM * C; i += FT) {
    const int u = i / C, ch = i % C;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (u < rows) {
      const int tok = tok0 + u / p.group, g = u % p.group;
      const float* q = static_cast<const float*>(p.q) + c.seq * p.q_seq + tok * p.q_token +
                       (static_cast<int64_t>(c.h) * p.group + g) * D;
      x = __ldg(reinterpret_cast<const float4*>(q) + ch);
    }
    const float sl = p.scale * LOG2E;
    *reinterpret_cast<float4*>(&sq[u][ch * 4]) = make_float4(x.x * sl, x.y * sl, x.z * sl, x.w * sl);
  }
}

// Cached rows [k0, k0 + FN) of K or V: those in [0, s1) and [w0, last], which are the rows that
// chunk_blocks_ok checked the table for; zeros for the others, which are not read.
template <int D>
__device__ __forceinline__ void load_rows(const AttnParams& p, const void* pool, int64_t base, const int32_t* trow, int k0,
                                          int s1, int w0, int last, float (*dst)[D + 4]) {
  constexpr int C = D / 4;
  for (int i = threadIdx.x; i < FN * C; i += FT) {
    const int u = i / C, ch = i % C;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    const int j = k0 + u;
    if (j <= last && (j < s1 || j >= w0))
      x = __ldg(reinterpret_cast<const float4*>(static_cast<const char*>(pool) + p.rows.row(base, trow, j)) + ch);
    *reinterpret_cast<float4*>(&dst[u][ch * 4]) = x;
  }
}

// Thread (ty, tx) = (t / 16, t % 16): logits of query rows 4 ty + a, cached rows tx + 16 b.
template <int D>
__device__ __forceinline__ void tile_logits(const float (*sq)[D + 4], const float (*sk)[D + 4], int ty, int tx, float (&x)[4][4]) {
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int b = 0; b < 4; ++b) x[a][b] = 0.f;
  for (int e = 0; e < D; e += 4) {
    float4 qa[4], kb[4];
#pragma unroll
    for (int a = 0; a < 4; ++a) qa[a] = *reinterpret_cast<const float4*>(&sq[4 * ty + a][e]);
#pragma unroll
    for (int b = 0; b < 4; ++b) kb[b] = *reinterpret_cast<const float4*>(&sk[tx + 16 * b][e]);
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        x[a][b] = fmaf(qa[a].x, kb[b].x, x[a][b]);
        x[a][b] = fmaf(qa[a].y, kb[b].y, x[a][b]);
        x[a][b] = fmaf(qa[a].z, kb[b].z, x[a][b]);
        x[a][b] = fmaf(qa[a].w, kb[b].w, x[a][b]);
      }
  }
}

}  // namespace
}  // namespace tri
