// attn_mass.cu -- the accumulated weight of every cached row under a chunk of
// queries: mass[j] += sum over the queries that see row j of e^(x_j - lse).
// A CTA owns cached rows and goes over the chunk's queries, so each mass is
// summed in a fixed order and written once, without atomics.
//
// Per pair of a query row (token, head) and a cached row it sees: 2 D flop and
// one exponential. Computed as S^T = K Q^T, cached rows on the lanes of tensor
// memory: a thread owns a cached row, the weights of a query column need only
// that column's lse, and the sum over queries is the thread's own.
//
// bf16 rows, tcgen05; a copy warp, an MMA warp, and four warpgroups that read S
// from four 128-column buffers of tensor memory and add up the weights:
//   - mass_few_kernel, at most FEW query tiles (an observation window): the
//     queries stay in shared memory and the cache streams past them; bound by
//     the keys' bytes. One CTA per SM takes an equal share of all slices' tiles,
//     whatever the slices' lengths. A warpgroup takes every fourth tile of rows.
//   - mass_many_kernel: two tiles of rows stay in shared memory and the query
//     tiles stream past them. Under causality early rows are seen by many
//     queries and late ones by few, so a CTA takes tile i and tile N - 1 - i. Two
//     warpgroups per tile of rows take alternate query tiles.
//
// fp32 rows (mass_kernel): CUDA cores, 64 x 64 tiles in shared memory.
#include <cuda_runtime.h>

#include "attn_tc.cuh"
#include "attn_tile.cuh"

namespace tri {
namespace {

// ---------------------------------------------------------------------------
// bf16 rows
// ---------------------------------------------------------------------------
constexpr int MT = 640;    // copy warp, MMA warp, lse warp, second MMA warp, four warpgroups
constexpr int FEW = 2;     // query tiles that stay in shared memory
constexpr int SLOTS = 16;  // lse rows kept by mass_few_kernel (see there)
constexpr int LSE_ROWS = 16;  // and by mass_many_kernel

// Which tensor maps the queries have. A map asks each stride to be a multiple of the one
// before it that holds the dimension between them, so (element, head, token, sequence) has
// tokens inside sequences, or the other way round, and a box of it is a column of a packed
// tile. Queries at other strides are rows by number, a box for each token's heads (weights of a
// 4096-token prompt: 298 us, by columns 76; a warp issues the boxes one lane at a time).
enum QueryOrder { Q_ROWS, Q_TOKENS_INSIDE, Q_SEQUENCES_INSIDE };
struct QueryDims {
  QueryOrder order;
  int64_t inner, outer;  // elements between tokens, or sequences: those of the inner dimension first
};
inline QueryDims query_dims(const AttnParams& p, int head_dim) {
  const int64_t token = static_cast<int64_t>(p.n_kv_heads) * p.group * head_dim, seqs = p.q_seq ? p.n_seq : 1;
  auto fits = [](int64_t outer, int64_t inner, int64_t n) { return outer % inner == 0 && outer / inner >= n; };
  if (p.n_q == 1 || seqs == 1) {  // (strides of dimensions of one are never used)
    const int64_t only = p.n_q > 1 ? p.q_token : seqs > 1 ? p.q_seq : token;
    if (!fits(only, head_dim, p.n_kv_heads * p.group)) return {Q_ROWS, 0, 0};
    return {Q_TOKENS_INSIDE, only, only * p.n_q};
  }
  if (fits(p.q_token, head_dim, p.n_kv_heads * p.group) && fits(p.q_seq, p.q_token, p.n_q)) return {Q_TOKENS_INSIDE, p.q_token, p.q_seq};
  if (fits(p.q_seq, head_dim, p.n_kv_heads * p.group) && fits(p.q_token, p.q_seq, seqs)) return {Q_SEQUENCES_INSIDE, p.q_seq, p.q_token};
  return {Q_ROWS, 0, 0};
}
inline bool encode_queries(RowMaps<false>& map, const AttnParams& p, int head_dim, const QueryDims& q, Encode encode) {
  const bool tokens_inside = q.order == Q_TOKENS_INSIDE;
  const cuuint64_t seqs = static_cast<cuuint64_t>(p.q_seq ? p.n_seq : 1), tokens = static_cast<cuuint64_t>(p.n_q);
  const cuuint32_t box_tokens = static_cast<cuuint32_t>(TROWS / p.group);
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(head_dim), static_cast<cuuint64_t>(p.n_kv_heads * p.group),
                              tokens_inside ? tokens : seqs, tokens_inside ? seqs : tokens};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(head_dim) * 2, static_cast<cuuint64_t>(q.inner) * 2,
                                 static_cast<cuuint64_t>(q.outer) * 2};
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(p.group), tokens_inside ? box_tokens : 1, tokens_inside ? 1 : box_tokens};
  const cuuint32_t step[4] = {1, 1, 1, 1};
  return encode(&map.m[0], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(p.q), dims, strides, box, step,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
inline bool encode_queries(RowMaps<true>& maps, const AttnParams& p, int head_dim, const QueryDims&, Encode encode) {
  const int64_t elements = (p.n_seq - 1) * p.q_seq + (p.n_q - 1) * p.q_token + static_cast<int64_t>(p.n_kv_heads) * p.group * head_dim;
  return encode_row_maps(maps, p.q, elements * 2, head_dim, p.group, encode);
}

// Query tiles [qt, qt + n) of a chunk into the tiles at dst, by one warp, arriving once on
// `bar`. Rows past the tokens of a tile's box, or of the chunk, are not written.
template <int D, bool QROWS>
__device__ __forceinline__ void load_queries_tma(uint32_t dst, const RowMaps<QROWS>& maps, bool tokens_inside, const AttnParams& p, const Chunk& c,
                                                 int qt, int n, uint64_t* bar, int lane) {
  constexpr int COLS = D / 64;
  const int tpt = TROWS / p.group, tok0 = qt * tpt;
  if constexpr (QROWS) {
    const int toks = min(n * tpt, c.n_new - tok0);
    if (lane == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(toks * p.group * D * 2));
    __syncwarp();
    for (int i = lane; i < toks * COLS; i += 32) {
      const int col = i % COLS, tok = i / COLS, tile = tok / tpt;
      const int64_t at = (c.seq * p.q_seq + (tok0 + tok) * p.q_token) / 8 + c.h * p.group * (D / 8);  // 16-byte units
      tma_load2(dst + (tile * COLS + col) * TCOL + (tok - tile * tpt) * p.group * 128, &maps.m[at % (D / 8)], 64 * col,
                static_cast<int>(at / (D / 8)), bar);
    }
  } else if (lane == 0) {
    const int seq = p.q_seq ? c.seq : 0;
    mbar_arrive_expect_tx(bar, static_cast<uint32_t>(n * tpt * p.group * D * 2));
    for (int i = 0; i < n; ++i) {
      const int tok = tok0 + i * tpt;
#pragma unroll
      for (int a = 0; a < COLS; ++a)
        tma_load4(dst + (i * COLS + a) * TCOL, &maps.m[0], 64 * a, c.h * p.group, tokens_inside ? tok : seq, tokens_inside ? seq : tok, bar);
    }
  }
}
// -lse in base 2 of a query tile's rows (-inf, so no weight, past its tokens), by
// a warp: row 32 k + lane in x[k].
__device__ __forceinline__ void get_lse(float (&x)[TROWS / 32], const AttnParams& p, const Chunk& c, int tpt, int qt, int lane) {
#pragma unroll
  for (int k = 0; k < TROWS / 32; ++k) {
    const int u = k * 32 + lane, tok = qt * tpt + u / p.group;
    const bool live = u < tpt * p.group && tok < c.n_new;
    x[k] = live ? -LOG2E * p.lse_in[c.seq * p.lse_seq + static_cast<int64_t>(tok) * (p.n_kv_heads * p.group) +
                                    c.h * p.group + u % p.group]
                : NEG_INF;
  }
}

// Columns of query tile qt that see cached row j: [lo, hi).
__device__ __forceinline__ void columns_seeing(const AttnParams& p, const Chunk& c, int tpt, int qt, int j, int& lo, int& hi) {
  const int tok0 = qt * tpt, toks = min(tpt, c.n_new - tok0), rf = c.r0 + tok0;
  lo = min(max(j - rf, 0), tpt) * p.group;
  int end = toks;
  if (p.window && j >= p.n_sink) end = static_cast<int>(min(static_cast<int64_t>(end), static_cast<int64_t>(j) + p.window - rf));
  hi = max(end, 0) * p.group;
}

// Sum of the weights of this thread's cached row over 64 query columns (of a
// tile's, from `first`) at ts; `done` runs when S has been read. ALL: every
// column counts, else columns [lo, hi) whatever the others hold. (Two loops: as
// one with selects the 4096-token prompt took 189 us
// where this took 164.)
template <bool ALL, class Done>
__device__ __forceinline__ float row_weights(uint32_t ts, const float* nl, int first, float sl, int lo, int hi, Done done) {
  float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
  uint32_t x[64];
  tmem_ld32(ts + first, x);
  tmem_ld32(ts + first + 32, x + 32);
  tmem_wait_ld();
  done();
#pragma unroll
  for (int k = 0; k < 64; k += 4) {
    const float4 n = *reinterpret_cast<const float4*>(nl + first + k);
    float e0, e1, e2, e3;
    fma2(e0, e1, __uint_as_float(x[k]), __uint_as_float(x[k + 1]), sl, n.x, n.y);
    fma2(e2, e3, __uint_as_float(x[k + 2]), __uint_as_float(x[k + 3]), sl, n.z, n.w);
    e0 = fast_exp2(e0);
    e1 = fast_exp2(e1);
    e2 = fast_exp2(e2);
    e3 = fast_exp2(e3);
    if constexpr (!ALL) {
      const unsigned c = first + k - lo, n_cols = hi > lo ? hi - lo : 0;
      e0 = c < n_cols ? e0 : 0.f;
      e1 = c + 1 < n_cols ? e1 : 0.f;
      e2 = c + 2 < n_cols ? e2 : 0.f;
      e3 = c + 3 < n_cols ? e3 : 0.f;
    }
    add2(s0, s1, e0, e1);
    add2(s2, s3, e2, e3);
  }
  return (s0 + s1) + (s2 + s3);
}
template <class Done>
__device__ __forceinline__ float row_weights(uint32_t ts, const float* nl, int first, float sl, bool all, int lo, int hi, Done done) {
  return all ? row_weights<true>(ts, nl, first, sl, 0, 0, done) : row_weights<false>(ts, nl, first, sl, lo, hi, done);
}

// Whether every query row of tile qt sees every row of the cached tile at k0.
__device__ __forceinline__ bool all_seen(const AttnParams& p, const Chunk& c, int tpt, int qt, int k0) {
  const int tok0 = qt * tpt, rf = c.r0 + tok0, rl = rf + tpt - 1;
  return tok0 + tpt <= c.n_new && k0 + TROWS - 1 <= rf &&
         (p.window == 0 || k0 + TROWS <= p.n_sink || k0 > rl - p.window);
}
__device__ __forceinline__ bool any_seen(const AttnParams& p, const Chunk& c, int tpt, int qt, int k0) {
  const int tok0 = qt * tpt;
  if (tok0 >= c.n_new) return false;
  const int rf = c.r0 + tok0, rl = rf + min(tpt, c.n_new - tok0) - 1;
  return tile_seen(p, k0, TROWS, max(rf, 0), rl);
}

// Zeros in the rows of `tiles` query tiles that their boxes do not write.
template <int D>
__device__ __forceinline__ void clear_tails(unsigned char* q, int tiles, int group) {
  const int first = TROWS / group * group;
  for (int i = threadIdx.x; i < tiles * (D / 64) * (TROWS - first) * 8; i += MT) {
    const int col = i / ((TROWS - first) * 8), rest = i % ((TROWS - first) * 8);
    *reinterpret_cast<uint4*>(q + col * TCOL + first * 128 + rest * 16) = make_uint4(0, 0, 0, 0);
  }
  fence_proxy_async_smem();
}

template <int D>
struct TcMass {
  static constexpr int TILE = D / 64 * TCOL;
  static constexpr int NST = D == 128 ? 4 : 8;
  static constexpr int RING = FEW * TILE;  // after the resident tiles
  static constexpr int CTRL = RING + NST * TILE;
  static constexpr int BYTES = CTRL + 256 + SLOTS * FEW * TROWS * 4;
  static_assert(BYTES <= 227 * 1024, "shared memory");
};
struct MassCtl {
  uint64_t full[8], empty[8];     // ring stages
  uint64_t res_full, res_free;    // the resident tiles have landed; are no longer read
  uint64_t s_full[4], s_free[4];  // S complete; read
  uint32_t tmem;
  int flag;
  int first_slice, first_tile;
  float nl[SLOTS][FEW][TROWS];    // -lse, base 2 (mass_many_kernel: LSE_ROWS rows, then the rows' sums)
};
static_assert(sizeof(MassCtl) <= 256 + SLOTS * FEW * TROWS * 4, "control block");

template <int D, bool ODD, bool QROWS>
__global__ void __launch_bounds__(MT, 1)
    mass_many_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ RowMaps<ODD> kmap,
                     const __grid_constant__ RowMaps<QROWS> qmap, const __grid_constant__ RowNumbers rn, bool tokens_inside) {
  using L = TcMass<D>;
  extern __shared__ __align__(1024) unsigned char smem[];
  MassCtl& ctl = *reinterpret_cast<MassCtl*>(smem + L::CTRL);
  const int t = threadIdx.x, w = __shfl_sync(FULL_MASK, t >> 5, 0), lane = t & 31;
  const int n_ls = p.n_seq * p.n_kv_heads, ls = blockIdx.x % n_ls, pair = blockIdx.x / n_ls;
  Chunk c;
  if (!chunk_of(p, ls, c)) return;
  const int r_end = c.n - 1;
  const int n_tiles = (c.n + TROWS - 1) / TROWS, other = n_tiles - 1 - pair;
  if (pair > other) return;
  const int nk = pair == other ? 1 : 2;
  const int32_t* trow = p.rows.seq_table(c.s);
  if (!chunk_blocks_ok(p, trow, c.r0, r_end, &ctl.flag)) return;
  const int tpt = TROWS / p.group, n_qt = __shfl_sync(FULL_MASK, (c.n_new + tpt - 1) / tpt, 0);
  auto k_of = [&](int kt) { return (kt ? other : pair) * TROWS; };
  // the query tiles that see any row of tile kt: [lo, hi) (uniform values, see prefill_tc_kernel)
  struct Range {
    int lo, hi;
    __device__ bool has(int i) const { return i >= lo && i < hi; }
  };
  auto range_of = [&](int kt) {
    Range r{0, 0};
    if (kt < nk) {
      // tokens from the tile's first row on, and with a window up to its last row + window - 1
      const int k0 = k_of(kt);
      r.lo = max(0, k0 - c.r0) / tpt;
      r.hi = n_qt;
      if (p.window && k0 >= p.n_sink) {
        const int64_t last = static_cast<int64_t>(k0) + TROWS - 1 + p.window - 1 - c.r0;
        r.hi = static_cast<int>(min(static_cast<int64_t>(n_qt), last < 0 ? 0 : last / tpt + 1));
      }
    }
    return Range{__shfl_sync(FULL_MASK, r.lo, 0), __shfl_sync(FULL_MASK, r.hi, 0)};
  };
  const Range need0 = range_of(0), need1 = range_of(1);

  if (t == 0) {
    for (int i = 0; i < L::NST; ++i) {
      mbar_init(&ctl.full[i], 2);    // the queries and their lse
      mbar_init(&ctl.empty[i], 2);   // two threads' MMAs
    }
    mbar_init(&ctl.res_full, nk);
    for (int b = 0; b < 4; ++b) {
      mbar_init(&ctl.s_full[b], 1);
      mbar_init(&ctl.s_free[b], 4);
    }
    mbar_init_fence();
  }
  clear_tails<D>(smem + L::RING, L::NST, p.group);
  if (w == 1) tmem_alloc(&ctl.tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = __shfl_sync(FULL_MASK, ctl.tmem, 0), res = smem_addr(smem), ring = res + L::RING;
  bool ok = true;

  if (w == 0) {
    const LaneBox<D> box(rn, lane);
    for (int kt = 0; kt < nk; ++kt) {
      const int blk = tile_block<D>(p, rn.box_rows, trow, c.seq, k_of(kt), c.n, lane);
      load_tile<D, ODD>(res + kt * L::TILE, kmap, box, box_place<D, ODD>(rn, box, blk, c.h, k_of(kt)), &ctl.res_full, lane);
    }
    int cnt = 0;
    for (int qt = 0; qt < n_qt && ok; ++qt) {
      if (!need0.has(qt) && !need1.has(qt)) continue;
      const int st = cnt % L::NST;
      if (cnt >= L::NST) ok = __all_sync(FULL_MASK, mbar_wait_bounded(&ctl.empty[st], (cnt / L::NST - 1) & 1));
      if (!ok) break;
      load_queries_tma<D, QROWS>(ring + st * L::TILE, qmap, tokens_inside, p, c, qt, 1, &ctl.full[st], lane);
      __syncwarp();
      ++cnt;
    }
    if (!ok && lane == 0) set_status(p.dev_status, TRI_DEV_TIMEOUT);
    // copies in flight finish before shared memory is given up
    (void)mbar_wait_bounded(&ctl.res_full, 0);
    for (int u = max(0, cnt - L::NST); u < cnt; ++u) (void)mbar_wait_bounded(&ctl.full[u % L::NST], (u / L::NST) & 1);
  } else if (w == 2) {
    // ---- lse: a tile's is loaded two tiles before it is stored (two register sets in turn) ----
    // Tile i's is in row i % LSE_ROWS, overwritten for tile i + 16 once the products of tile
    // i + 16 - NST are done, at least eight after those of tile i. Product p + 8 goes to p's
    // buffer and waits until its warpgroup has read product p + 4, so is done with p.
    static_assert(LSE_ROWS - L::NST >= 8, "lse rows");
    const int per_tile = tpt * p.n_kv_heads * p.group;
    const float* src[TROWS / 32];
    int tok[TROWS / 32];  // within a tile; n_new: none
#pragma unroll
    for (int k = 0; k < TROWS / 32; ++k) {
      const int u = k * 32 + lane;
      tok[k] = u < tpt * p.group ? u / p.group : c.n_new;
      src[k] = p.lse_in + c.seq * p.lse_seq + static_cast<int64_t>(u / p.group) * (p.n_kv_heads * p.group) + c.h * p.group + u % p.group;
    }
    auto next = [&](int qt) {
      while (qt < n_qt && !need0.has(qt) && !need1.has(qt)) ++qt;
      return qt;
    };
    auto get = [&](float (&x)[TROWS / 32], int qt) {
#pragma unroll
      for (int k = 0; k < TROWS / 32; ++k)
        x[k] = qt < n_qt && qt * tpt + tok[k] < c.n_new ? __ldg(src[k] + static_cast<int64_t>(qt) * per_tile) : -NEG_INF;
    };
    uint32_t cnt = 0;
    auto store = [&](const float (&x)[TROWS / 32]) {
      const uint32_t st = cnt % L::NST;
      if (cnt >= L::NST) ok = __all_sync(FULL_MASK, mbar_wait_bounded(&ctl.empty[st], (cnt / L::NST - 1) & 1));
#pragma unroll
      for (int k = 0; k < TROWS / 32; ++k) (&ctl.nl[0][0][0])[cnt % LSE_ROWS * TROWS + k * 32 + lane] = -LOG2E * x[k];
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.full[st]);
      ++cnt;
    };
    float xa[TROWS / 32], xb[TROWS / 32];
    int qa = next(0), qb = next(qa + 1);
    get(xa, qa);
    get(xb, qb);
    while (qa < n_qt && ok) {
      store(xa);
      qa = next(qb + 1);
      get(xa, qa);
      if (qb >= n_qt || !ok) break;
      store(xb);
      qb = next(qa + 1);
      get(xb, qb);
    }
    if (!ok && lane == 0) set_status(p.dev_status, TRI_DEV_TIMEOUT);
  } else if (w < 4) {
    // ---- MMAs: products w == 1 ? 0, 2, .. : 1, 3, .. ----
    const int par = w == 1 ? 0 : 1;
    if (elect_one()) {
      constexpr uint32_t IDESC = bf16_idesc(TROWS, TROWS, false);
      constexpr uint64_t STAGE = L::TILE >> 4;  // (descriptors count 16 bytes)
      const uint64_t dk = sw128_desc(res), dr = sw128_desc(ring);
      uint32_t cnt = 0, n = 0;  // stages taken, products counted
      ok = mbar_wait_bounded(&ctl.res_full, 0);
      for (int qt = 0; qt < n_qt && ok; ++qt) {
        const bool need[2] = {need0.has(qt), need1.has(qt)};
        if (!need[0] && !need[1]) continue;
        const uint32_t st = cnt % L::NST;
        ok = mbar_wait_bounded(&ctl.full[st], (cnt / L::NST) & 1);
#pragma unroll
        for (int kt = 0; kt < 2; ++kt) {
          if (!need[kt] || !ok) continue;
          if ((n & 1) == par) {
            const uint32_t b = n & 3;
            // (the phase before an mbarrier's first counts as complete)
            ok = mbar_wait_bounded(&ctl.s_free[b], ((n >> 2) + 1) & 1);
            if (!ok) continue;
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              const uint64_t off = (k >> 2) * (TCOL >> 4) + (k & 3) * 2;
              umma_f16(tm + b * 128, dk + kt * STAGE + off, dr + st * STAGE + off, IDESC, k > 0);
            }
            umma_commit(&ctl.s_full[b]);
          }
          ++n;
        }
        if (!ok) break;
        umma_commit(&ctl.empty[st]);
        ++cnt;
      }
      if (!ok) set_status(p.dev_status, TRI_DEV_TIMEOUT);
    }
    __syncwarp();
  } else {
    // ---- weights: warpgroup g takes products g, g + 4, .., which are in buffer g ----
    const uint32_t g = (w - 4) >> 2;
    const int u = t & 127;
    const uint32_t ts = tm + g * 128 + (static_cast<uint32_t>((w & 3) * 32) << 16);
    const float sl = p.scale * LOG2E;
    float sums[2] = {0.f, 0.f};
    uint32_t cnt = 0, n = 0;
    for (int qt = 0; qt < n_qt && ok; ++qt) {
      const bool need[2] = {need0.has(qt), need1.has(qt)};
      if (!need[0] && !need[1]) continue;
#pragma unroll
      for (int kt = 0; kt < 2; ++kt) {
        if (!need[kt] || !ok) continue;
        if ((n & 3) == g) {
          // (the product was issued once the tile's lse were there too)
          ok = __all_sync(FULL_MASK, mbar_wait_bounded(&ctl.s_full[g], (n >> 2) & 1));
          if (!ok) continue;
          tc_fence_after();
          const int k0 = k_of(kt);
          const bool all = all_seen(p, c, tpt, qt, k0);
          int lo = 0, hi = TROWS;
          if (!all) columns_seeing(p, c, tpt, qt, k0 + u, lo, hi);
          const float* nl = &ctl.nl[0][0][0] + cnt % LSE_ROWS * TROWS;
          sums[kt] += row_weights(ts, nl, 0, sl, all, lo, hi, [] {});
          sums[kt] += row_weights(ts, nl, 64, sl, all, lo, hi, [&] {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl.s_free[g]);
          });
        }
        ++n;
      }
      ++cnt;
    }
    if (!ok && lane == 0) set_status(p.dev_status, TRI_DEV_TIMEOUT);
#pragma unroll
    for (int kt = 0; kt < 2; ++kt) ctl.nl[8 + kt * 4 + g][0][u] = sums[kt];  // (the ring's lse rows are below)
  }
  tc_fence_before();
  const bool fine = __syncthreads_and(ok);
  tc_fence_after();
  if (w == 1) tmem_dealloc(tm, 512);
  if (fine && t < nk * TROWS) {
    const int kt = t / TROWS, u = t % TROWS, j = k_of(kt) + u;
    const float(*part)[FEW][TROWS] = ctl.nl + 8 + kt * 4;
    const float sum = (part[0][0][u] + part[1][0][u]) + (part[2][0][u] + part[3][0][u]);
    if (j <= r_end && sum != 0.f) p.mass[c.s * p.n_cap + j] += sum;
  }
}

// Tiles of rows of a slice that hold any (none of one with a bad count).
__device__ __forceinline__ int tiles_of(const AttnParams& p, int ls) {
  const int seq = ls / p.n_kv_heads;
  const int n = p.n_valid[slice_of(p, seq, ls - seq * p.n_kv_heads)];
  if (n >= 0 && n <= p.n_cap) return (n + TROWS - 1) / TROWS;
  set_status(p.dev_status, TRI_DEV_NVALID_OVER_CAP);
  return 0;
}

// Where the CTA's share of all tiles starts, and how many it has: (by the CTA;
// sums of the slices before each thread's run of slices, then a walk).
__device__ __forceinline__ int64_t my_share(const AttnParams& p, MassCtl& ctl) {
  __shared__ int64_t warp_sum[MT / 32];
  const int n_ls = p.n_seq * p.n_kv_heads, t = threadIdx.x;
  const int per = (n_ls + MT - 1) / MT, s0 = min(n_ls, t * per), s1 = min(n_ls, s0 + per);
  int64_t mine = 0;
  for (int s = s0; s < s1; ++s) mine += tiles_of(p, s);
  int64_t upto = mine;
#pragma unroll
  for (int k = 1; k < 32; k <<= 1) {
    const int64_t x = __shfl_up_sync(FULL_MASK, upto, k);
    if ((t & 31) >= k) upto += x;
  }
  if ((t & 31) == 31) warp_sum[t >> 5] = upto;
  __syncthreads();
  int64_t total = 0;
  for (int i = 0; i < MT / 32; ++i) {
    if (i < (t >> 5)) upto += warp_sum[i];
    total += warp_sum[i];
  }
  const int64_t x0 = total * blockIdx.x / gridDim.x, x1 = total * (blockIdx.x + 1) / gridDim.x;
  int64_t base = upto - mine;
  if (x0 >= base && x0 < upto) {
    for (int s = s0; s < s1; ++s) {
      const int n = tiles_of(p, s);
      if (x0 < base + n) {
        ctl.first_slice = s;
        ctl.first_tile = static_cast<int>(x0 - base);
        break;
      }
      base += n;
    }
  }
  __syncthreads();
  return x1 - x0;
}

// Every block that some query of the chunk sees rows of is in the pool (by a warp).
__device__ __forceinline__ bool warp_blocks_ok(const AttnParams& p, const Chunk& c, int lane) {
  const int32_t* trow = p.rows.seq_table(c.s);
  if (!trow) return true;
  const Visible first = visible_rows(max(c.r0, 0), p.n_sink, p.window);
  const int s1 = visible_rows(c.n - 1, p.n_sink, p.window).s1;
  bool ok = true;
  for (int b = lane; b <= (c.n - 1) >> p.rows.block_shift; b += 32) {
    const int r = b << p.rows.block_shift;
    if (r >= s1 && r + p.rows.block_size <= first.w0) continue;
    const int v = __ldg(trow + b);
    ok = ok && v >= 0 && v < p.rows.num_blocks;
  }
  return __all_sync(FULL_MASK, ok);
}

// The queries of one (sequence, KV head) and a run of its tiles of rows: a
// segment. Segments follow each other; every role walks them alike.
//
// The lse rows of segment g are in slot g % SLOTS. A warpgroup that still reads
// them when segment g + SLOTS is loaded would have to be a tile more than 12
// tiles behind the MMAs, and S's four buffers let it fall back by at most 8.
template <int D, bool ODD, bool QROWS>
__global__ void __launch_bounds__(MT, 1)
    mass_few_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ RowMaps<ODD> kmap,
                    const __grid_constant__ RowMaps<QROWS> qmap, const __grid_constant__ RowNumbers rn, bool tokens_inside) {
  using L = TcMass<D>;
  extern __shared__ __align__(1024) unsigned char smem[];
  MassCtl& ctl = *reinterpret_cast<MassCtl*>(smem + L::CTRL);
  const int t = threadIdx.x, w = __shfl_sync(FULL_MASK, t >> 5, 0), lane = t & 31;
  const int64_t share = my_share(p, ctl);
  if (share == 0) return;
  const int tpt = TROWS / p.group;

  if (t == 0) {
    for (int i = 0; i < L::NST; ++i) {
      mbar_init(&ctl.full[i], 1);
      mbar_init(&ctl.empty[i], 1);
    }
    mbar_init(&ctl.res_full, 1);
    mbar_init(&ctl.res_free, 1);
    for (int b = 0; b < 4; ++b) {
      mbar_init(&ctl.s_full[b], 1);
      mbar_init(&ctl.s_free[b], 4);
    }
    mbar_init_fence();
  }
  clear_tails<D>(smem, FEW, p.group);
  if (w == 1) tmem_alloc(&ctl.tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = __shfl_sync(FULL_MASK, ctl.tmem, 0), res = smem_addr(smem), ring = res + L::RING;
  bool ok = true;

  // The walk, by a whole warp: body(segment, chunk, query tiles, cached tile k0) for
  // every tile of the share that some query sees; next(segment, chunk, query tiles)
  // before its first and last(segment) after its last one.
  auto walk = [&](auto&& next, auto&& body, auto&& last) {
    int ls = ctl.first_slice, first = ctl.first_tile, seg = 0;
    for (int64_t left = share; left > 0 && ok; ++ls, first = 0) {
      const int n = tiles_of(p, ls);
      if (n == 0) continue;
      const int end = static_cast<int>(min(static_cast<int64_t>(n), first + left));
      left -= end - first;
      Chunk c;
      if (!chunk_of(p, ls, c)) continue;
      if (!warp_blocks_ok(p, c, lane)) {
        if (lane == 0) set_status(p.dev_status, TRI_DEV_BAD_BLOCK);
        continue;
      }
      const TileList list = tiles_seen(p, max(c.r0, 0), c.n - 1);
      const int a = min(end, list.a), b = max(first, list.b), e = min(end, list.e);
      if (first >= a && b >= e) continue;
      const int n_qt = __shfl_sync(FULL_MASK, (c.n_new + tpt - 1) / tpt, 0);
      next(seg, c, n_qt);
      for (int i = first; i < a && ok; ++i) body(seg, c, n_qt, i * TROWS);
      for (int i = b; i < e && ok; ++i) body(seg, c, n_qt, i * TROWS);
      if (ok) last(seg);
      ++seg;
    }
  };

  if (w == 0) {
    int cnt = 0, segs = 0;
    const int32_t* trow = nullptr;
    int blk = 0, blk_row = -1;  // (of the row it is for)
    const LaneBox<D> box(rn, lane);
    walk(
        [&](int seg, const Chunk& c, int n_qt) {
          if (seg > 0) ok = __all_sync(FULL_MASK, mbar_wait_bounded(&ctl.res_free, (seg - 1) & 1));
          if (!ok) return;
          for (int qt = 0; qt < n_qt; ++qt) {
            float x[TROWS / 32];
            get_lse(x, p, c, tpt, qt, lane);
#pragma unroll
            for (int k = 0; k < TROWS / 32; ++k) ctl.nl[seg % SLOTS][qt][k * 32 + lane] = x[k];
          }
          __syncwarp();
          load_queries_tma<D, QROWS>(res, qmap, tokens_inside, p, c, 0, n_qt, &ctl.res_full, lane);
          segs = seg + 1;
          trow = p.rows.seq_table(c.s);
          blk_row = -1;
        },
        [&](int, const Chunk& c, int, int k0) {
          const int st = cnt % L::NST;
          if (blk_row != k0) blk = tile_block<D>(p, rn.box_rows, trow, c.seq, k0, c.n, lane);
          const Place place = box_place<D, ODD>(rn, box, blk, c.h, k0);
          // (the next tile's is on its way while this one waits for its stage)
          blk_row = k0 + TROWS;
          const int blk_next = tile_block<D>(p, rn.box_rows, trow, c.seq, blk_row, c.n, lane);
          if (cnt >= L::NST) ok = __all_sync(FULL_MASK, mbar_wait_bounded(&ctl.empty[st], (cnt / L::NST - 1) & 1));
          if (!ok) return;
          load_tile<D, ODD>(ring + st * L::TILE, kmap, box, place, &ctl.full[st], lane);
          blk = blk_next;
          ++cnt;
        },
        [](int) {});
    if (!ok && lane == 0) set_status(p.dev_status, TRI_DEV_TIMEOUT);
    // copies in flight finish before shared memory is given up
    if (segs) (void)mbar_wait_bounded(&ctl.res_full, (segs - 1) & 1);
    for (int u = max(0, cnt - L::NST); u < cnt; ++u) (void)mbar_wait_bounded(&ctl.full[u % L::NST], (u / L::NST) & 1);
  } else if (w == 1) {
    // (lane 0 issues: what a commit covers is its own thread's MMAs)
    constexpr uint32_t IDESC = bf16_idesc(TROWS, TROWS, false);
    constexpr uint64_t STAGE = L::TILE >> 4;  // (descriptors count 16 bytes)
    const uint64_t dq = sw128_desc(res), dr = sw128_desc(ring);
    int cnt = 0;
    uint32_t used = 0;  // 8 bits per buffer: uses so far, mod 256
    walk([&](int seg, const Chunk&, int) { ok = __all_sync(FULL_MASK, mbar_wait_bounded(&ctl.res_full, seg & 1)); },
         [&](int, const Chunk& c, int n_qt, int k0) {
           const int st = cnt % L::NST, b = cnt & 3;
           ok = __all_sync(FULL_MASK, mbar_wait_bounded(&ctl.full[st], (cnt / L::NST) & 1));
           uint32_t n = (used >> (8 * b)) & 255u;
           for (int qt = 0; qt < n_qt && ok; ++qt) {
             if (!any_seen(p, c, tpt, qt, k0)) continue;
             // (the phase before an mbarrier's first counts as complete)
             ok = __all_sync(FULL_MASK, mbar_wait_bounded(&ctl.s_free[b], (n - 1) & 1));
             if (!ok) break;
             tc_fence_after();
             if (lane == 0) {
#pragma unroll
               for (int k = 0; k < D / 16; ++k) {
                 const uint64_t off = (k >> 2) * (TCOL >> 4) + (k & 3) * 2;
                 umma_f16(tm + b * 128, dr + st * STAGE + off, dq + qt * STAGE + off, IDESC, k > 0);
               }
               umma_commit(&ctl.s_full[b]);
             }
             __syncwarp();
             ++n;
           }
           used = (used & ~(255u << (8 * b))) | ((n & 255u) << (8 * b));
           if (ok && lane == 0) umma_commit(&ctl.empty[st]);
           ++cnt;
         },
         [&](int) {
           if (lane == 0) umma_commit(&ctl.res_free);
         });
    if (!ok && lane == 0) set_status(p.dev_status, TRI_DEV_TIMEOUT);
    __syncwarp();
  } else if (w >= 4) {
    const int b = (w - 4) >> 2, u = t & 127;
    const uint32_t ts = tm + b * 128 + (static_cast<uint32_t>((w & 3) * 32) << 16);
    const float sl = p.scale * LOG2E;
    int cnt = 0, n = 0;
    walk([](int, const Chunk&, int) {},
         [&](int seg, const Chunk& c, int n_qt, int k0) {
           if ((cnt++ & 3) != b) return;
           const int j = k0 + u;
           float* mass = p.mass + c.s * p.n_cap + j;
           const float old = j < c.n ? *mass : 0.f;  // (on its way while the products run)
           float sum = 0.f;
           for (int qt = 0; qt < n_qt && ok; ++qt) {
             if (!any_seen(p, c, tpt, qt, k0)) continue;
             ok = __all_sync(FULL_MASK, mbar_wait_bounded(&ctl.s_full[b], n & 1));
             if (!ok) break;
             ++n;
             tc_fence_after();
             const bool all = all_seen(p, c, tpt, qt, k0);
             int lo = 0, hi = TROWS;
             if (!all) columns_seeing(p, c, tpt, qt, j, lo, hi);
             sum += row_weights(ts, ctl.nl[seg % SLOTS][qt], 0, sl, all, lo, hi, [] {});
             sum += row_weights(ts, ctl.nl[seg % SLOTS][qt], 64, sl, all, lo, hi, [&] {
               tc_fence_before();
               __syncwarp();
               if (lane == 0) mbar_arrive(&ctl.s_free[b]);
             });
           }
           if (ok && j < c.n && sum != 0.f) *mass = old + sum;
         },
         [](int) {});
    if (!ok && lane == 0) set_status(p.dev_status, TRI_DEV_TIMEOUT);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (w == 1) tmem_dealloc(tm, 512);
}

template <int D, bool ODD, bool QROWS>
cudaError_t launch_tc(const AttnParams& p, const RowNumbers& rn, const QueryDims& qd, cudaStream_t st) {
  RowMaps<ODD> kmap;
  RowMaps<QROWS> qmap;
  const Encode encode = tensor_map_encode();
  if (!encode || !encode_rows(kmap, p.k, p, D, rn, encode) || !encode_queries(qmap, p, D, qd, encode)) return cudaErrorInvalidValue;
  const int tpt = TROWS / p.group, n_qt = (p.n_q + tpt - 1) / tpt;
  const bool few = n_qt <= FEW;
  auto kern = few ? mass_few_kernel<D, ODD, QROWS> : mass_many_kernel<D, ODD, QROWS>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, TcMass<D>::BYTES);
  if (e != cudaSuccess) return e;
  const int64_t n_ls = static_cast<int64_t>(p.n_seq) * p.n_kv_heads, tiles = (p.n_cap + TROWS - 1) / TROWS;
  const int64_t ctas = few ? min(static_cast<int64_t>(SMS), n_ls * tiles) : n_ls * ((tiles + 1) / 2);
  if (ctas > 0x7fffffff) return cudaErrorInvalidValue;
  kern<<<static_cast<unsigned>(ctas), MT, TcMass<D>::BYTES, st>>>(p, kmap, qmap, rn, qd.order == Q_TOKENS_INSIDE);
  note_launch();
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_bf16(const AttnParams& p, cudaStream_t st) {
  RowNumbers rn{};
  if (!row_numbers(p, rn)) return cudaErrorNotSupported;
  const QueryDims qd = query_dims(p, D);
  if (qd.order == Q_ROWS) {
    if ((p.n_seq - 1) * p.q_seq + (p.n_q - 1) * p.q_token > static_cast<int64_t>(0x7fffffff - 2 * TROWS) * D) return cudaErrorNotSupported;
    return rn.odd ? launch_tc<D, true, true>(p, rn, qd, st) : launch_tc<D, false, true>(p, rn, qd, st);
  }
  return rn.odd ? launch_tc<D, true, false>(p, rn, qd, st) : launch_tc<D, false, false>(p, rn, qd, st);
}

// ---------------------------------------------------------------------------
// fp32 rows
// ---------------------------------------------------------------------------
template <int D>
struct MassSmem {
  float q[FM][D + 4];
  float k[FN][D + 4];
  float lse2[FM];
  float part[16][FN];
  int flag;
};

template <int D>
__global__ void __launch_bounds__(FT) mass_kernel(const __grid_constant__ AttnParams p, int n_tiles) {
  extern __shared__ __align__(16) unsigned char raw[];
  MassSmem<D>& sm = *reinterpret_cast<MassSmem<D>*>(raw);
  const int ls = blockIdx.x / n_tiles, k0 = blockIdx.x % n_tiles * FN;
  const int t = threadIdx.x, ty = t / 16, tx = t % 16, G = p.group;
  Chunk c;
  if (!chunk_of(p, ls, c)) return;
  const int r_end = c.r0 + c.n_new - 1;
  if (!tile_seen(p, k0, FN, max(c.r0, 0), r_end)) return;
  const int64_t base = p.rows.slice_base(c.s);
  const int32_t* trow = p.rows.seq_table(c.s);
  const int last = min(k0 + FN - 1, r_end);
  // (with a bad entry for rows that some query sees the whole slice is left out, by each of its CTAs)
  if (!chunk_blocks_ok(p, trow, c.r0, r_end, &sm.flag)) return;
  const int s1 = visible_rows(max(r_end, 0), p.n_sink, p.window).s1, w0 = visible_rows(max(c.r0, 0), p.n_sink, p.window).w0;
  load_rows<D>(p, p.k, base, trow, k0, s1, w0, last, sm.k);
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
  const int tpt = FM / G;
  for (int tok0 = 0; tok0 < c.n_new; tok0 += tpt) {
    const int toks = min(tpt, c.n_new - tok0), rows = toks * G, r_first = c.r0 + tok0;
    if (!tile_seen(p, k0, FN, max(r_first, 0), r_first + toks - 1)) continue;
    __syncthreads();
    load_queries<D>(p, c, tok0, rows, sm.q);
    if (t < rows)
      sm.lse2[t] = LOG2E * p.lse_in[c.seq * p.lse_seq + static_cast<int64_t>(tok0 + t / G) * (p.n_kv_heads * G) + c.h * G + t % G];
    __syncthreads();
    float x[4][4];
    tile_logits<D>(sm.q, sm.k, ty, tx, x);
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const int u = 4 * ty + a;
      if (u >= rows) continue;
      const int r = r_first + u / G;
#pragma unroll
      for (int b = 0; b < 4; ++b)
        if (sees(p, r, k0 + tx + 16 * b)) sum[b] += fast_exp2(x[a][b] - sm.lse2[u]);
    }
  }
#pragma unroll
  for (int b = 0; b < 4; ++b) sm.part[ty][tx + 16 * b] = sum[b];
  __syncthreads();
  if (t < FN && k0 + t <= last) {
    float w = 0.f;
    for (int i = 0; i < 16; ++i) w += sm.part[i][t];
    p.mass[c.s * p.n_cap + k0 + t] += w;
  }
}

template <int D>
cudaError_t launch_fp32(const AttnParams& p, cudaStream_t st) {
  auto kern = mass_kernel<D>;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(sizeof(MassSmem<D>)));
  if (e != cudaSuccess) return e;
  const int n_tiles = (p.n_cap + FN - 1) / FN;
  const int64_t ctas = static_cast<int64_t>(p.n_seq) * p.n_kv_heads * n_tiles;
  if (ctas > 0x7fffffff) return cudaErrorInvalidValue;
  kern<<<static_cast<unsigned>(ctas), FT, sizeof(MassSmem<D>), st>>>(p, n_tiles);
  note_launch();
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_mass(const AttnParams& p, tri_dtype dt, int head_dim, cudaStream_t st) {
  if (dt == TRI_BF16) return head_dim == 64 ? launch_bf16<64>(p, st) : launch_bf16<128>(p, st);
  return head_dim == 64 ? launch_fp32<64>(p, st) : launch_fp32<128>(p, st);
}

}  // namespace tri
