// attn_prefill.cu -- causal attention of a chunk of new tokens over the cache,
// optionally windowed with first rows that stay visible.
//
// The group's query heads share a KV head's rows, so a query row is a (token,
// head) pair and a tile packs 128 of them. Per pair of a query row and a cached
// row it sees: 4 D flop and one exponential.
//
// bf16 rows (prefill_tc_kernel): tcgen05, one CTA per SM with two query tiles.
// A step takes 64 cached rows: S = Q K^T (128 x 64), weights P from S, O += P V.
// One step is a chain -- eight MMAs and their completion 1056 clocks, then the
// weights, then a signal back, about 250 clocks -- several times longer than
// its MMAs run, so two steps of each query tile are in flight, each in its own
// buffer of tensor memory. (With one 128-row step per query tile in flight the
// 8192-token prompt took 419 us at 55% of the tensor cores' cycles.) Roles:
//   - the copy warp brings the cache's 128-row tiles of K and V, in turn, into a
//     ring by TMA (a pool's blocks as boxes of a tile);
//   - an MMA warp per query tile: one thread issues, step by step, the product
//     with V once the weights are ready and the S of the step after next (issuing
//     blocks for as long as the MMAs run);
//   - two warpgroups per query tile turn S into P: a thread has 32 of a query
//     row's columns (row = lane of tensor memory), and two threads share their
//     row's maximum through shared memory. P, rounded to bf16, takes its part of
//     S's place as the A operand of the product with V, so the weights never
//     pass through shared memory.
// Tensor memory: per query tile 2 x 64 columns of S/P and D columns of O.
// The running maximum of a row is raised only when a step exceeds it by more
// than 8 (a factor of 256): O is then rescaled in tensor memory, once the
// products before have completed; until then weights are up to 256, which costs
// no precision in a floating format.
// A few CTAs' worth of queries (a follow-up question on a long cache) would leave
// most SMs idle: then a cluster of CTAs shares a pair of query tiles, each takes a
// run of the cached rows, and they join through their shared memories. The
// tensor cores are not what bounds such a call, so the weights go in as a bf16 pair
// (p rounded, and the rest rounded) instead of rounded once. In a large call the pair would
// cost a third of the time (8192-token prompt 380 -> 505 us, 8 prompts at d 64 with a window 175
// -> 206) for an rms error of 1.11e-4 instead of 1.47e-4, of which the output's own bf16
// rounding is 1.11e-4: there p is rounded once.
// Steps at the edge of what the rows see are masked by position; rows of V past
// the last query's are set to zero in shared memory, whatever they hold.
//
// fp32 rows (prefill_kernel): CUDA cores, 64 x 64 tiles in shared memory.
#include <cuda_runtime.h>

#include "attn_tc.cuh"
#include "attn_tile.cuh"

namespace tri {
namespace {

// ---------------------------------------------------------------------------
// bf16 rows
// ---------------------------------------------------------------------------
constexpr int STEP = 64;     // cached rows of a step
constexpr float RAISE = 8.f;
constexpr int MAX_SPLITS = 8;  // CTAs that share query tiles

template <int D, int NQ>
struct TcSmem {
  static constexpr int TILE = D / 64 * TCOL;
  static constexpr int THREADS = 128 + NQ * 256;  // copy warp, two MMA warps, an idle one, two warpgroups per query tile
  static constexpr int NST = D == 128 ? 4 : 5;
  static constexpr int RING = NQ * TILE;  // after the query tiles
  static constexpr int TMEM = NQ * 256;   // columns: per query tile 2 x 64 of S/P and up to 128 of O
  static constexpr int CTRL = RING + NST * TILE;
  static constexpr int BYTES = CTRL + 4608;
  static_assert(BYTES <= 227 * 1024, "shared memory");
};

struct TcCtl {
  uint64_t full[8], empty[8];                           // ring stages
  uint64_t q_ready[2];                                  // the query tile is in shared memory
  uint64_t s_full[2][2], p_ready[2][2], o_ready[2][2];  // [query tile][half of a tile of rows]: S complete; P written; its product complete
  uint64_t v_fix;                                       // the last tile of V has landed, before its tail is cleared
  uint32_t tmem;
  int flag[2];                                          // a bad table entry for rows that the query tile sees
  float mx[2][2][2][TROWS];                             // maxima: [step parity][query tile][half][row]
};
static_assert(sizeof(TcCtl) <= 4608, "control block");

__device__ __forceinline__ float max_of(const uint32_t (&x)[32]) {
  float m[4];  // (four chains)
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    m[k] = __uint_as_float(x[k]);
#pragma unroll
    for (int e = 4; e < 28; e += 8) m[k] = max3(m[k], __uint_as_float(x[e + k]), __uint_as_float(x[e + 4 + k]));
    m[k] = fmaxf(m[k], __uint_as_float(x[28 + k]));
  }
  return fmaxf(max3(m[0], m[1], m[2]), m[3]);
}
// N columns of this thread's row of O, times a.
template <int N>
__device__ __forceinline__ void scale_o(uint32_t to, float a) {
#pragma unroll
  for (int k = 0; k < N / 16; ++k) {
    uint32_t o[16];
    tmem_ld16(to + k * 16, o);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * a);
    tmem_st16(to + k * 16, o);
  }
}
// Weights 2^(x sl - mu) of 32 columns, rounded to bf16 (hi), with PAIR also what the
// rounding left (lo); returns their fp32 sum.
template <bool PAIR>
__device__ __forceinline__ float weights_of(const uint32_t (&x)[32], float sl, float mu, uint32_t (&hi)[16], uint32_t (&lo)[16]) {
  float l0 = 0.f, l1 = 0.f, l2 = 0.f, l3 = 0.f;
#pragma unroll
  for (int k = 0; k < 16; k += 2) {
    float e0, e1, e2, e3;
    fma2(e0, e1, __uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1]), sl, -mu);
    fma2(e2, e3, __uint_as_float(x[2 * k + 2]), __uint_as_float(x[2 * k + 3]), sl, -mu);
    e0 = fast_exp2(e0);
    e1 = fast_exp2(e1);
    e2 = fast_exp2(e2);
    e3 = fast_exp2(e3);
    add2(l0, l1, e0, e1);
    add2(l2, l3, e2, e3);
    hi[k] = pack_bf16(e0, e1);
    hi[k + 1] = pack_bf16(e2, e3);
    if constexpr (PAIR) {
      lo[k] = pack_bf16(e0 - bf16_lo(hi[k]), e1 - bf16_hi(hi[k]));
      lo[k + 1] = pack_bf16(e2 - bf16_lo(hi[k + 1]), e3 - bf16_hi(hi[k + 1]));
    }
  }
  return (l0 + l1) + (l2 + l3);
}

template <int D, int NQ, bool FEW_CTAS, bool ODD>
__global__ void __launch_bounds__((TcSmem<D, NQ>::THREADS), 3 - NQ)
    prefill_tc_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ RowMaps<ODD> kmap,
                      const __grid_constant__ RowMaps<ODD> vmap, const __grid_constant__ RowNumbers rn, int n_tiles, int cluster) {
  using L = TcSmem<D, NQ>;
  const int splits = FEW_CTAS ? cluster : 1;
  extern __shared__ __align__(1024) unsigned char smem[];  // (the swizzle goes by address)
  TcCtl& ctl = *reinterpret_cast<TcCtl*>(smem + L::CTRL);
  // (values that the MMA warps use come through a shuffle, so that the compiler
  // knows them to be the same in a warp and keeps them in uniform registers)
  const int t = threadIdx.x, w = __shfl_sync(FULL_MASK, t >> 5, 0), lane = t & 31, G = p.group;
  // the last tokens see the most rows: their tiles first
  const int n_ls = p.n_seq * p.n_kv_heads;
  const int unit = static_cast<int>(blockIdx.x) / splits, rank = static_cast<int>(blockIdx.x) % splits;
  const int ls = unit % n_ls, tile = n_tiles - 1 - unit / n_ls;
  Chunk c;
  if (!chunk_of(p, ls, c)) return;  // (all returns here are a whole cluster's)
  const int tpt = TROWS / G;  // tokens per query tile
  const int tok0 = tile * NQ * tpt;
  if (tok0 >= c.n_new) return;
  const int toks0 = min(tpt, c.n_new - tok0), toks1 = NQ == 2 ? min(tpt, c.n_new - tok0 - toks0) : 0;
  const int nq = toks1 > 0 ? 2 : 1;
  const int rf0 = c.r0 + tok0, rl0 = rf0 + toks0 - 1;
  const int rf1 = rl0 + 1, rl1 = rl0 + toks1;  // (empty when nq is 1)
  const int r_hi = rl1;
  const int32_t* trow = p.rows.seq_table(c.s);
  const TileList list = tiles_seen(p, rf0, r_hi);
  // this CTA's run of the list: tiles first .. first + n_list - 1
  const int first = __shfl_sync(FULL_MASK, list.count() * rank / splits, 0);
  const int n_list = __shfl_sync(FULL_MASK, list.count() * (rank + 1) / splits - first, 0);
  // the steps (row / 64) that some row of query tile q sees: below e, and below a or from f on
  struct Steps {
    int a, f, e;
    __device__ bool has(int x) const { return x < e && (x < a || x >= f); }
  };
  auto steps_of = [&](int q) {
    const int rf = q ? rf1 : rf0, rl = q ? rl1 : rl0;
    const int a = p.window ? (min(p.n_sink, max(rl + 1, 0)) + STEP - 1) / STEP : 0;
    const int f = p.window ? max(0, max(rf, 0) - p.window + 1) / STEP : 0;
    return Steps{__shfl_sync(FULL_MASK, a, 0), __shfl_sync(FULL_MASK, f, 0), __shfl_sync(FULL_MASK, rl < 0 ? 0 : rl / STEP + 1, 0)};
  };
  auto tile_row = [&](int i) { return list.at(first + i) * TROWS; };

  if (t == 0) {
    for (int i = 0; i < L::NST; ++i) {
      mbar_init(&ctl.full[i], 1);
      mbar_init(&ctl.empty[i], nq);
    }
    for (int q = 0; q < 2; ++q) {
      mbar_init(&ctl.q_ready[q], 8);  // (a warp arrives once)
      for (int b = 0; b < 2; ++b) {
        mbar_init(&ctl.s_full[q][b], 1);
        mbar_init(&ctl.p_ready[q][b], 8);
        mbar_init(&ctl.o_ready[q][b], 1);
      }
    }
    mbar_init(&ctl.v_fix, 1);
    ctl.flag[0] = ctl.flag[1] = 0;
    mbar_init_fence();
  }
  if (w == 1) tmem_alloc(&ctl.tmem, L::TMEM);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = __shfl_sync(FULL_MASK, ctl.tmem, 0);
  auto s_col = [&](int q, int b) { return tm + (q * 2 + b) * STEP; };
  auto o_col = [&](int q) { return tm + (NQ + q) * 128; };
  const uint32_t qa = smem_addr(smem), ring = qa + L::RING;
  bool ok = true;
  float m = NEG_INF, l = 0.f;  // (weights' threads: running maximum and sum; steps done)
  int n = 0;

  if (w == 0) {
    // ---- copies: K and V tiles take the ring's stages in turn ----
    // (A pool's tables are checked as they are read: a query tile with a bad entry for rows
    // that it sees is left out. Its flag is set before the rows are brought, and by no other
    // rows, so a query tile that is done with its rows reads it settled. Boxes that no query
    // sees are zeros: they may have no block any more.)
    int cnt = 0;
    uint32_t bad = 0;  // bit q
    int see0[NQ], see1[NQ];
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      see0[q] = visible_rows(max(q ? rf1 : rf0, 0), p.n_sink, p.window).w0;
      see1[q] = visible_rows(max(q ? rl1 : rl0, 0), p.n_sink, p.window).s1;
    }
    auto block_of = [&](int k0) {
      if (!trow) return c.seq;
      const int row = k0 + lane / (D / 64) * rn.box_rows;
      uint32_t seen = 0;
#pragma unroll
      for (int q = 0; q < NQ; ++q)
        if (q < nq && row <= (q ? rl1 : rl0) && (row < see1[q] || row + rn.box_rows > see0[q])) seen |= 1u << q;
      if (!seen || row >= k0 + TROWS) return p.rows.num_blocks;
      const int blk = tile_block<D>(p, rn.box_rows, trow, c.seq, k0, c.n, lane);
      if (blk == p.rows.num_blocks) bad |= seen;
      return blk;
    };
    const LaneBox<D> box(rn, lane);
    auto place_of = [&](int blk, int k0) { return box_place<D, ODD>(rn, box, blk, c.h, k0); };
    int blk_next = n_list ? block_of(tile_row(0)) : 0;
    Place place = n_list ? place_of(blk_next, tile_row(0)) : Place{0, 0};
    for (; cnt < 2 * n_list && ok; ++cnt) {
      const int st = cnt % L::NST, k0 = tile_row(cnt >> 1);
      if (!(cnt & 1) && cnt + 2 < 2 * n_list)  // (on its way while this tile waits for its stage)
        blk_next = block_of(tile_row((cnt >> 1) + 1));
      if (cnt >= L::NST) ok = __all_sync(FULL_MASK, mbar_wait_bounded(&ctl.empty[st], (cnt / L::NST - 1) & 1));
      if (!ok) break;
      const bool is_v = cnt & 1;
      const bool fix = is_v && k0 + TROWS - 1 > r_hi;
      uint64_t* bar = fix ? &ctl.v_fix : &ctl.full[st];
      if (bad & 1) ctl.flag[0] = 1;
      if (bad & 2) ctl.flag[1] = 1;
      __syncwarp();
      load_tile<D, ODD>(ring + st * L::TILE, is_v ? vmap : kmap, box, place, bar, lane);
      if (is_v && cnt + 1 < 2 * n_list) place = place_of(blk_next, tile_row((cnt >> 1) + 1));
      if (fix) {
        ok = __all_sync(FULL_MASK, mbar_wait_bounded(&ctl.v_fix, 0));
        if (!ok) break;
        unsigned char* v = smem + L::RING + st * L::TILE;
        for (int i = (r_hi + 1 - k0) * 8 + lane; i < TROWS * 8; i += 32)
#pragma unroll
          for (int a = 0; a < D / 64; ++a) *reinterpret_cast<uint4*>(v + a * TCOL + i * 16) = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.full[st]);
      }
    }
    if (bad) set_status(p.dev_status, TRI_DEV_BAD_BLOCK);
    if (!ok && lane == 0) {
      set_status(p.dev_status, TRI_DEV_TIMEOUT);
      // let the copies in flight finish before shared memory is given up
      for (int u = max(0, cnt - L::NST); u < cnt; ++u) (void)mbar_wait_bounded(&ctl.full[u % L::NST], (u / L::NST) & 1);
    }
  } else if (w < 3) {
    // ---- MMAs of query tile w - 1 ----
    const int q = w - 1;
    const Steps need = steps_of(q);
    if (q < nq && elect_one()) {
      constexpr uint32_t IQK = bf16_idesc(TROWS, STEP, false), IPV = bf16_idesc(TROWS, D, true);
      constexpr uint64_t STAGE = L::TILE >> 4;  // (descriptors count 16 bytes)
      const uint64_t dq = sw128_desc(qa + q * L::TILE), dk = sw128_desc(ring), dv = sw128_desc_mn(ring);
      const uint32_t to = o_col(q);
      auto issue_s = [&](uint32_t at, int b) {
        const uint64_t ds = dk + at * STAGE + b * (STEP * 8);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint64_t off = (k >> 2) * (TCOL >> 4) + (k & 3) * 2;
          umma_f16(s_col(q, b), dq + off, ds + off, IQK, k > 0);
        }
        umma_commit(&ctl.s_full[q][b]);
      };
      uint32_t use[2] = {0, 0};  // products of each buffer
      auto step_of = [&](int i) { return 2 * list.at(first + i); };
      ok = mbar_wait_bounded(&ctl.q_ready[q], 0);
      if (n_list > 0 && ok) {
        ok = mbar_wait_bounded(&ctl.full[0], 0);
        tc_fence_after();
#pragma unroll
        for (int b = 0; b < 2; ++b)
          if (ok && need.has(step_of(0) + b)) issue_s(0, b);
        umma_commit(&ctl.empty[0]);
      }
      for (int i = 0; i < n_list && ok; ++i) {
        const bool more = i + 1 < n_list;
        const int x = step_of(i), xn = more ? step_of(i + 1) : need.e;
        const uint32_t cv = 2 * i + 1, sv = cv % L::NST, sk = (cv + 1) % L::NST;
        ok = mbar_wait_bounded(&ctl.full[sv], (cv / L::NST) & 1);
        if (ok && more) ok = mbar_wait_bounded(&ctl.full[sk], ((cv + 1) / L::NST) & 1);
        if (!ok) break;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          if (need.has(x + b)) {
            ok = ok && mbar_wait_bounded(&ctl.p_ready[q][b], use[b] & 1);
            tc_fence_after();
            // P's rows 16 j .. 16 j + 15 of the step sit at columns 32 (j / 2) + 8 (j % 2) of its buffer
            const uint64_t ds = dv + sv * STAGE + b * (STEP * 8);
            umma_ts(to, s_col(q, b), ds, IPV, use[0] + use[1] > 0);
#pragma unroll
            for (int j = 1; j < STEP / 16; ++j) umma_ts(to, s_col(q, b) + (j >> 1) * 32 + (j & 1) * 8, ds + j * 128, IPV, true);
            if constexpr (FEW_CTAS) {  // the pair's second half, 16 columns on
#pragma unroll
              for (int j = 0; j < STEP / 16; ++j) umma_ts(to, s_col(q, b) + 16 + (j >> 1) * 32 + (j & 1) * 8, ds + j * 128, IPV, true);
            }
            umma_commit(&ctl.o_ready[q][b]);
            ++use[b];
          }
          if (need.has(xn + b)) issue_s(sk, b);
        }
        umma_commit(&ctl.empty[sv]);
        if (more) umma_commit(&ctl.empty[sk]);
      }
      if (!ok) set_status(p.dev_status, TRI_DEV_TIMEOUT);
    }
    __syncwarp();
  } else if (w >= 4 && (w < 12 || nq == 2)) {
    // ---- weights: thread u of a half = query row u of tile q, 32 columns of a step ----
    const int q = (w - 4) >> 3, half = ((w - 4) >> 2) & 1, u = t & 127;
    const int toks = q ? toks1 : toks0, rows = toks * G, rf = q ? rf1 : rf0, rl = q ? rl1 : rl0;
    load_query_tile<D, 256>(qa + q * L::TILE, p, c.seq, c.h, tok0 + q * tpt, rows, half * 128 + u);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&ctl.q_ready[q]);
    const uint32_t lanes = static_cast<uint32_t>((w & 3) * 32) << 16;
    const uint32_t to = o_col(q) + half * (D / 2) + lanes;
    const int r = rf + u / G;
    const int pair = 1 + q * 4 + (w & 3);  // named barrier of the two warps of 32 rows
    const float sl = p.scale * LOG2E;
    const Steps need = steps_of(q);
    uint32_t par = 0;         // bit b: parity of buffer b's next use
    int last = 0;             // the last step's buffer, and the parity of that use
    uint32_t last_par = 0;
    // The products of all steps before are complete. (Those before the last one are: S of
    // this step was issued after them.)
    auto wait_products = [&] {
      if (n > 0 && ok) ok = __all_sync(FULL_MASK, mbar_wait_bounded(&ctl.o_ready[q][last], last_par));
      tc_fence_after();
    };
    for (int step = 0; step < 2 * n_list; ++step) {
      const int b = step & 1;
      if (!need.has(2 * list.at(first + (step >> 1)) + b)) continue;
      const uint32_t ts = s_col(q, b) + half * 32 + lanes;
      // (after a wait that gave up the loop runs on without waiting, since the
      // two halves meet at barriers)
      if (ok) ok = __all_sync(FULL_MASK, mbar_wait_bounded(&ctl.s_full[q][b], (par >> b) & 1));
      tc_fence_after();
      uint32_t x[32];
      tmem_ld32(ts, x);
      tmem_wait_ld();
      const int k0 = tile_row(step >> 1) + b * STEP;
      const bool inner = k0 + STEP - 1 <= rf && (p.window == 0 || k0 > rl - p.window || k0 + STEP <= p.n_sink);
      if (!inner) {
        const uint32_t bits = seen_bits(p, r, k0, half);
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if (!(bits & (1u << e))) x[e] = 0xff800000u;  // -inf
      }
      float mx = max_of(x);
      ctl.mx[n & 1][q][half][u] = mx;
      asm volatile("bar.sync %0, 64;" ::"r"(pair) : "memory");
      mx = fmaxf(mx, ctl.mx[n & 1][q][half ^ 1][u]) * sl;
      if (n == 0) {
        m = mx;
      } else if (__any_sync(FULL_MASK, mx > m + RAISE)) {  // (the same in both halves)
        const float mn = fmaxf(m, mx);
        const float a = mn == NEG_INF ? 1.f : fast_exp2(m - mn);
        m = mn;
        l *= a;
        wait_products();
        scale_o<D / 2>(to, a);
      }
      const float mu = m == NEG_INF ? 0.f : m;
      uint32_t hi[16], lo[16];
      l += weights_of<FEW_CTAS>(x, sl, mu, hi, lo);
      tmem_st16(ts, hi);
      if constexpr (FEW_CTAS) tmem_st16(ts + 16, lo);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.p_ready[q][b]);
      last = b;
      last_par = (par >> b) & 1;
      par ^= 1u << b;
      ++n;
    }
    wait_products();
    // (without a step nothing has waited for the other warps' copies of the query tile)
    if (n == 0 && ok) ok = __all_sync(FULL_MASK, mbar_wait_bounded(&ctl.q_ready[q], 0));
    ctl.mx[n & 1][q][half][u] = l;
    asm volatile("bar.sync %0, 64;" ::"r"(pair) : "memory");
    const float l_half = ctl.mx[n & 1][q][half ^ 1][u];
    l = half ? l_half + l : l + l_half;
    if (!ok) {
      if (lane == 0) set_status(p.dev_status, TRI_DEV_TIMEOUT);
    } else if (!FEW_CTAS && !ctl.flag[q]) {
      const float inv = l != 0.f ? 1.f / l : 0.f;
      // The rows go out through the query tile, which no product reads any more (the last
      // product's completion is that of every MMA of the query tile): stored
      // by the thread that holds them, each warp's 32 rows then leave as whole 16-byte
      // chunks of D bytes a row (a thread storing its own row touches 32 bytes of memory
      // for each 16 it writes).
      unsigned char* stage = smem + q * L::TILE;
      constexpr int CHUNKS = D / 16;  // of a thread's half row
      auto chunk_at = [&](int row, int k) {
        const int ch = half * CHUNKS + k;
        return reinterpret_cast<uint4*>(stage + (ch >> 3) * TCOL + row * 128 + (((ch & 7) ^ (row & 7)) << 4));
      };
#pragma unroll
      for (int k = 0; k < D / 64; ++k) {
        uint32_t o[32];
        if (n > 0) {
          tmem_ld32(to + k * 32, o);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0u;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t y[4];
#pragma unroll
          for (int f = 0; f < 4; ++f)
            y[f] = pack_bf16(__uint_as_float(o[8 * e + 2 * f]) * inv, __uint_as_float(o[8 * e + 2 * f + 1]) * inv);
          *chunk_at(u, k * 4 + e) = make_uint4(y[0], y[1], y[2], y[3]);
        }
      }
      __syncwarp();
      auto head_of = [&](int row) {
        const int tok = row / G;
        return (static_cast<int64_t>(c.seq) * p.n_q + tok0 + q * tpt + tok) * (p.n_kv_heads * G) + c.h * G + row - tok * G;
      };
#pragma unroll
      for (int i = 0; i < CHUNKS; ++i) {
        const int row = (w & 3) * 32 + i * (32 / CHUNKS) + lane / CHUNKS, k = lane % CHUNKS;
        if (row < rows)
          *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + head_of(row) * D + (half * CHUNKS + k) * 8) = *chunk_at(row, k);
      }
      const int64_t head = head_of(u);
      if (p.lse && half == 0 && u < rows) p.lse[head] = l != 0.f ? LN2 * (m + log2f(l)) : NEG_INF;
    }
  }
  tc_fence_before();
  __syncthreads();  // (nothing uses the tiles in shared memory any more)
  tc_fence_after();
  if constexpr (FEW_CTAS) {
    // ---- join: every CTA's sums go to its shared memory, and each joins its share of rows ----
    constexpr int RS = D + 4;  // floats of a row (16-byte stores of neighbouring rows in other banks)
    static_assert(NQ * TROWS * RS * 4 <= L::CTRL, "the rows' sums");
    float* so = reinterpret_cast<float*>(smem);
    float* sm = &ctl.mx[0][0][0][0];  // m and l of 256 rows
    if (w >= 4 && (w < 12 || nq == 2)) {
      const int q = (w - 4) >> 3, half = ((w - 4) >> 2) & 1, u = t & 127, row = q * TROWS + u;
      const uint32_t to = o_col(q) + half * (D / 2) + (static_cast<uint32_t>((w & 3) * 32) << 16);
#pragma unroll
      for (int k = 0; k < D / 32; ++k) {
        uint32_t o[16];
        if (n > 0) {
          tmem_ld16(to + k * 16, o);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = 0u;
        }
#pragma unroll
        for (int e = 0; e < 16; e += 4)
          *reinterpret_cast<uint4*>(so + row * RS + half * (D / 2) + k * 16 + e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
      }
      if (half == 0) {
        sm[row] = m;
        sm[256 + row] = ok && !ctl.flag[q] ? l : -1.f;
      }
    }
    cluster_sync(splits);
    const int n_rows = NQ * TROWS / splits;
    // the factors of a row's sums, 2^(m_k - m) / l, by a thread per row (-1: left out)
    float* factor = sm + 512;
    auto live = [&](int row) { return (row & 127) < (row >= TROWS ? toks1 : toks0) * G; };
    auto out_row = [&](int row) {
      return (static_cast<int64_t>(c.seq) * p.n_q + tok0 + (row >> 7) * tpt + (row & 127) / G) * (p.n_kv_heads * G) + c.h * G +
             (row & 127) % G;
    };
    if (t < n_rows) {
      const int row = rank * n_rows + t;
      float mk[MAX_SPLITS], lk[MAX_SPLITS], mj = NEG_INF, lj = 0.f;
#pragma unroll
      for (int k = 0; k < MAX_SPLITS; ++k) {
        mk[k] = k < splits ? cluster_ld(sm + row, k, splits) : NEG_INF;
        lk[k] = k < splits ? cluster_ld(sm + 256 + row, k, splits) : 0.f;
        mj = fmaxf(mj, mk[k]);
      }
      const float mu = mj == NEG_INF ? 0.f : mj;
      bool skip = false;
#pragma unroll
      for (int k = 0; k < MAX_SPLITS; ++k) {
        skip |= lk[k] < 0.f;
        mk[k] = fast_exp2(mk[k] - mu);
        lj = fmaf(lk[k], mk[k], lj);
      }
      const float inv = lj != 0.f ? 1.f / lj : 0.f;
#pragma unroll
      for (int k = 0; k < MAX_SPLITS; ++k)
        if (k < splits) factor[k * n_rows + t] = skip ? -1.f : mk[k] * inv;
      if (p.lse && !skip && live(row)) p.lse[out_row(row)] = lj != 0.f ? LN2 * (mj + log2f(lj)) : NEG_INF;
    }
    __syncthreads();
    for (int i = t; i < n_rows * (D / 4); i += L::THREADS) {
      const int r_own = i / (D / 4), row = rank * n_rows + r_own, e = i % (D / 4) * 4;
      if (!live(row) || factor[r_own] < 0.f) continue;
      float4 x[MAX_SPLITS];
#pragma unroll
      for (int k = 0; k < MAX_SPLITS; ++k)
        if (k < splits) x[k] = cluster_ld4(reinterpret_cast<const float4*>(so + row * RS + e), k, splits);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < MAX_SPLITS; ++k) {
        if (k >= splits) break;
        const float a = factor[k * n_rows + r_own];
        o.x = fmaf(x[k].x, a, o.x);
        o.y = fmaf(x[k].y, a, o.y);
        o.z = fmaf(x[k].z, a, o.z);
        o.w = fmaf(x[k].w, a, o.w);
      }
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + out_row(row) * D + e) =
          make_uint2(pack_bf16(o.x, o.y), pack_bf16(o.z, o.w));
    }
    cluster_sync(splits);  // a CTA's shared memory stays until the others have read it
  }
  if (w == 1) tmem_dealloc(tm, L::TMEM);
}

template <int D, bool ODD>
cudaError_t launch_tc(const AttnParams& p, const RowNumbers& rn, cudaStream_t st) {
  RowMaps<ODD> kmap, vmap;
  const Encode encode = tensor_map_encode();
  if (!encode || !encode_rows(kmap, p.k, p, D, rn, encode) || !encode_rows(vmap, p.v, p, D, rn, encode)) return cudaErrorInvalidValue;
  // one or two query tiles per CTA: at d 64 two CTAs with a tile each fit an SM, and one's
  // start and end hide behind the other's work (8 padded prompts of up to 4096 tokens, sinks
  // and a window of 1000: 189 us, with two tiles per CTA 199)
  constexpr int NQ = D == 128 ? 2 : 1;
  const int tokens = NQ * (TROWS / p.group), n_tiles = (p.n_q + tokens - 1) / tokens;
  const int64_t units = static_cast<int64_t>(p.n_seq) * p.n_kv_heads * n_tiles;
  if (units > 0x7fffffff) return cudaErrorInvalidValue;
  // CTAs per pair of query tiles: as many as the SMs have room for, with two tiles of rows each at least
  int64_t rows = p.n_cap;
  if (p.window) rows = min(rows, static_cast<int64_t>(p.window) + tokens + p.n_sink);
  const bool few = units * 2 <= SMS;
  int splits = 1;
  while (few && splits < MAX_SPLITS && units * splits * 2 <= SMS && rows >= 2 * splits * 2 * TROWS) splits *= 2;
  auto kern = few ? prefill_tc_kernel<D, NQ, true, ODD> : prefill_tc_kernel<D, NQ, false, ODD>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, TcSmem<D, NQ>::BYTES);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(units * splits));
  cfg.blockDim = dim3(TcSmem<D, NQ>::THREADS);
  cfg.dynamicSmemBytes = TcSmem<D, NQ>::BYTES;
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = static_cast<unsigned>(splits);
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = splits > 1;
  const cudaError_t r = cudaLaunchKernelEx(&cfg, kern, p, kmap, vmap, rn, n_tiles, splits);
  if (r == cudaSuccess) note_launch();
  return r;
}

// ---------------------------------------------------------------------------
// fp32 rows
// ---------------------------------------------------------------------------
template <int D>
struct PrefillSmem {
  float q[FM][D + 4];
  float k[FN][D + 4];
  float v[FN][D + 4];
  float w[FM][FN + 4];
  int flag;
};

template <int D>
__global__ void __launch_bounds__(FT) prefill_kernel(const __grid_constant__ AttnParams p, int n_tiles) {
  extern __shared__ __align__(16) unsigned char raw[];
  PrefillSmem<D>& sm = *reinterpret_cast<PrefillSmem<D>*>(raw);
  const int ls = blockIdx.x / n_tiles, tile = blockIdx.x % n_tiles;
  const int t = threadIdx.x, ty = t / 16, tx = t % 16, G = p.group;
  Chunk c;
  if (!chunk_of(p, ls, c)) return;
  const int tpt = FM / G;  // tokens per tile
  const int tok0 = tile * tpt;
  if (tok0 >= c.n_new) return;
  const int toks = min(tpt, c.n_new - tok0), rows = toks * G;
  const int r_first = c.r0 + tok0, r_last = r_first + toks - 1;
  const int64_t base = p.rows.slice_base(c.s);
  const int32_t* trow = p.rows.seq_table(c.s);
  if (!chunk_blocks_ok(p, trow, r_first, r_last, &sm.flag)) return;
  const int s1 = visible_rows(max(r_last, 0), p.n_sink, p.window).s1, w0 = visible_rows(max(r_first, 0), p.n_sink, p.window).w0;
  load_queries<D>(p, c, tok0, rows, sm.q);
  float m[4], l[4], o[4][D / 16];
  int r[4];
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    m[a] = NEG_INF;
    l[a] = 0.f;
    r[a] = r_first + (4 * ty + a) / G;
#pragma unroll
    for (int e = 0; e < D / 16; ++e) o[a][e] = 0.f;
  }
  for (int k0 = 0; k0 <= r_last; k0 += FN) {
    if (!tile_seen(p, k0, FN, r_first, r_last)) continue;
    __syncthreads();
    load_rows<D>(p, p.k, base, trow, k0, s1, w0, r_last, sm.k);
    load_rows<D>(p, p.v, base, trow, k0, s1, w0, r_last, sm.v);
    __syncthreads();
    float x[4][4];
    tile_logits<D>(sm.q, sm.k, ty, tx, x);
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      float mx = m[a];
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        if (!sees(p, r[a], k0 + tx + 16 * b)) x[a][b] = NEG_INF;
        mx = fmaxf(mx, x[a][b]);
      }
#pragma unroll
      for (int w = 8; w >= 1; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(FULL_MASK, mx, w));
      const float mu = mx == NEG_INF ? 0.f : mx;
      const float scale = fast_exp2(m[a] - mu);
      m[a] = mx;
      float sum = 0.f;
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const float w = fast_exp2(x[a][b] - mu);
        sum += w;
        sm.w[4 * ty + a][tx + 16 * b] = w;
      }
#pragma unroll
      for (int w = 8; w >= 1; w >>= 1) sum += __shfl_xor_sync(FULL_MASK, sum, w);
      l[a] = fmaf(l[a], scale, sum);
#pragma unroll
      for (int e = 0; e < D / 16; ++e) o[a][e] *= scale;
    }
    __syncthreads();
    for (int j = 0; j < FN; ++j) {
      float w[4];
#pragma unroll
      for (int a = 0; a < 4; ++a) w[a] = sm.w[4 * ty + a][j];
#pragma unroll
      for (int e = 0; e < D / 16; ++e) {
        const float vx = sm.v[j][tx + 16 * e];
#pragma unroll
        for (int a = 0; a < 4; ++a) o[a][e] = fmaf(w[a], vx, o[a][e]);
      }
    }
  }
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    const int u = 4 * ty + a;
    if (u >= rows) continue;
    const int64_t head = (static_cast<int64_t>(c.seq) * p.n_q + tok0 + u / G) * (p.n_kv_heads * G) + c.h * G + u % G;
    const float inv = l[a] != 0.f ? 1.f / l[a] : 0.f;
#pragma unroll
    for (int e = 0; e < D / 16; ++e) static_cast<float*>(p.out)[head * D + tx + 16 * e] = o[a][e] * inv;
    if (p.lse && tx == 0) p.lse[head] = l[a] != 0.f ? LN2 * (m[a] + log2f(l[a])) : NEG_INF;
  }
}

template <int D>
cudaError_t launch_fp32(const AttnParams& p, cudaStream_t st) {
  auto kern = prefill_kernel<D>;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(sizeof(PrefillSmem<D>)));
  if (e != cudaSuccess) return e;
  const int tpt = FM / p.group, n_tiles = (p.n_q + tpt - 1) / tpt;
  const int64_t ctas = static_cast<int64_t>(p.n_seq) * p.n_kv_heads * n_tiles;
  if (ctas > 0x7fffffff) return cudaErrorInvalidValue;
  kern<<<static_cast<unsigned>(ctas), FT, sizeof(PrefillSmem<D>), st>>>(p, n_tiles);
  note_launch();
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_prefill(const AttnParams& p, tri_dtype dt, int head_dim, cudaStream_t st) {
  if (dt == TRI_BF16) {
    RowNumbers rn{};
    if (!row_numbers(p, rn)) return cudaErrorNotSupported;
    if (head_dim == 64) return rn.odd ? launch_tc<64, true>(p, rn, st) : launch_tc<64, false>(p, rn, st);
    return rn.odd ? launch_tc<128, true>(p, rn, st) : launch_tc<128, false>(p, rn, st);
  }
  return head_dim == 64 ? launch_fp32<64>(p, st) : launch_fp32<128>(p, st);
}

}  // namespace tri
