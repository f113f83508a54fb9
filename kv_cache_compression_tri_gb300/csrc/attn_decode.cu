// attn_decode.cu -- attention of one new token per sequence over the cache,
// split over its length and joined, with the rows' accumulated weights.
//
// Per slice and query head g: x_j = scale * (q_g . k_j) over the visible rows,
// out_g = sum_j 2^(x_j - m) v_j / sum_j 2^(x_j - m). A slice's visible rows are
// cut into n_split runs, one CTA each; a run keeps a running maximum m, sum l and
// vector sum o per head (o and l rescaled when m grows). Joining takes the
// largest m of a head's runs, and the runs' l and o times 2^(m_run - m). Masses
// need every row's weight under the final log-sum, so the logits are left in
// the workspace and turned into weights after the join.
//
// Two ways to join. Up to MAX_CLUSTER runs of a slice form one thread-block
// cluster: each run's sums stay in its shared memory, the CTAs read each
// other's, each writes its share of the heads' elements and adds its own rows'
// masses -- one launch. More runs (few slices, long rows) write their sums to
// the workspace, and a second kernel, launched early and waiting for the first
// on the device, joins them.
//
// Bound: K and V are read once, 4 G flop per 4 bytes of a bf16 row pair: HBM.
//
// bf16 rows (decode_tiles_kernel). At most 8 query heads share a row, so the
// products are thin: one 16 x 8 x 16 warp MMA takes 16 rows against the
// group's heads. (A tcgen05 MMA takes at least 64 rows of M, and its
// operands and result would cross shared and tensor memory and two barriers
// per tile for a product that is not what bounds the kernel.) Each warp owns a
// ring of NST tiles of TK rows, filled with 16-byte asynchronous copies NST - 1
// tiles ahead, so no CTA barrier stands in the loop and a row never sits in
// registers while it is on its way. Rows out of sight are zero-filled by the
// copy and never read. In shared memory the 16-byte chunk c of row r lies at
// chunk c ^ (r & 7), so the eight rows of a matrix load hit eight different
// groups of banks.
//   S = K Q^T: A = 16 rows of K, B = the heads (registers, loaded once). A
//   thread gets rows g, g + 8 and heads 2t, 2t + 1 (g = lane / 4, t = lane % 4);
//   maxima and sums over rows are shuffles over g.
//   O^T += V^T P^T: A = V transposed by the matrix load, B = the weights of 16
//   rows, which a warp transpose turns from S's layout into B's. A head's
//   column of O^T and of S sit in the same threads, so rescaling is local. The
//   weights go in as a bf16 pair (p rounded, and the rest rounded): the product
//   carries 16 bits of them, at the cost of eight more MMAs that the memory
//   traffic hides.
//
// fp32 rows (decode_rows_kernel): the same rings, 8 lanes per row on the CUDA
// cores, fp32 throughout (a tensor-core product would drop the rows to 10 bits).
#include <cuda_runtime.h>

#include "attn_common.cuh"

namespace tri {
namespace {

// Row counts of a slice; false: nothing to do (faults are reported).
struct Run {
  int64_t s;       // slice of the cache
  int n, seq, h;   // valid rows, sequence, KV head
  int tok0, news;  // a chunk's pass: its tokens; n is then the rows that the last of them sees to,
  int first;       // and the first one's row (may be negative)
  Visible vis;     // (of a pass: to some token of it)
  int count;       // visible rows
};

// CHUNK (4-bit rows): the slice numbers count a chunk's passes.
template <bool CHUNK = false>
__device__ __forceinline__ bool slice_run(const AttnParams& p, int ls, Run& r) {
  int pass = 0;
  if constexpr (CHUNK) {
    pass = ls % p.passes;
    ls /= p.passes;
  }
  r.seq = ls / p.n_kv_heads;
  r.h = ls - r.seq * p.n_kv_heads;
  r.s = slice_of(p, r.seq, r.h);
  r.n = p.n_valid[r.s];
  const int nn = new_tokens(p, r.seq);
  if (r.n < 0 || r.n > p.n_cap) {
    set_status(p.dev_status, TRI_DEV_NVALID_OVER_CAP);
    return false;
  }
  if (nn <= 0) return false;
  if constexpr (CHUNK) {
    r.tok0 = pass * p.pass_tokens;
    r.news = min(p.pass_tokens, nn - r.tok0);
    if (r.news <= 0) return false;
    r.first = r.n - nn + r.tok0;
    r.n = max(r.first + r.news, 0);
    r.vis = visible_rows(r.n - 1, p.n_sink, p.window);
    r.vis.w0 = visible_rows(max(r.first, 0), p.n_sink, p.window).w0;
    r.vis.s1 = min(r.vis.s1, r.vis.w0);
  } else {
    r.vis = visible_rows(r.n - 1, p.n_sink, p.window);
  }
  r.count = r.vis.s1 + r.n - r.vis.w0;
  return true;
}

// ---------------------------------------------------------------------------
// bf16 rows
// ---------------------------------------------------------------------------
constexpr int NW = 4;  // warps per CTA
constexpr int MAX_CLUSTER = 16;  // (above 8 a kernel has to allow for it; a GPC of this GPU holds 16 such CTAs)

template <typename T, int D>
struct TileGeo {
  static constexpr int ROW = D * static_cast<int>(sizeof(T));  // bytes
  static constexpr int TK = 4096 / ROW;       // rows per tile: 4 KB of K and of V
  static constexpr int CH = ROW / 16;         // 16-byte chunks per row
  static constexpr int RPI = 32 / CH;         // rows per copy instruction of a warp
  static constexpr int TILE = TK * ROW;       // bytes of one tensor's tile
  static constexpr int NST = 2;
  static constexpr int WARP_RING = NST * 2 * TILE;
  static constexpr int SMEM = NW * WARP_RING;
  static constexpr int RUN = TK < 16 ? TK : 16;  // rows of a tile that lie in one block of any pool
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The row of out and lse that column g of a slice has, or -1 (a token that is not there).
template <bool CHUNK>
__device__ __forceinline__ int64_t row_of_column(const AttnParams& p, const Run& r, int g) {
  if (!CHUNK) return (static_cast<int64_t>(r.seq) * p.n_kv_heads + r.h) * p.group + g;
  const int tok = g / p.token_heads;
  if (tok >= r.news) return -1;
  return ((static_cast<int64_t>(r.seq) * p.n_q + r.tok0 + tok) * p.n_kv_heads + r.h) * p.token_heads + g - tok * p.token_heads;
}
// The result of a head's element, or of its log-sum, from the sums of all its rows.
template <typename T, int D, bool CHUNK>
__device__ __forceinline__ void store_out(const AttnParams& p, const Run& r, int g, int e, float o, float l) {
  const int64_t row = row_of_column<CHUNK>(p, r, g);
  if (!CHUNK || row >= 0) static_cast<T*>(p.out)[row * D + e] = from_f32<T>(l != 0.f ? o / l : 0.f);
}
template <bool CHUNK>
__device__ __forceinline__ void store_lse(const AttnParams& p, const Run& r, int g, float m, float l) {
  const int64_t row = row_of_column<CHUNK>(p, r, g);
  if (p.lse && (!CHUNK || row >= 0)) p.lse[row] = l != 0.f ? LN2 * (m + log2f(l)) : NEG_INF;
}

// mass[j] += sum over the heads of 2^(x_j - m) / l for rows j = row_at(i), i in
// [i0, i1) (-1: none), with the heads' joined m and l. A thread takes MASS_BATCH
// rows at a time, all loads before the first store: one by one, the load of a
// mass waits for the store before it (64 x 8 slices of up to 2176 rows: 66 us).
constexpr int MASS_BATCH = 8;
template <class RowAt>
__device__ __forceinline__ void add_masses(const AttnParams& p, const Run& r, int ls, const float* m, const float* l,
                                           int i0, int i1, RowAt row_at) {
  const int G = p.group;
  const float* logits = p.logits + static_cast<int64_t>(ls) * p.n_cap * G;
  float* mass = p.mass + r.s * p.n_cap;
  float lse2[MAX_GROUP];
#pragma unroll
  for (int g = 0; g < MAX_GROUP; ++g)  // (no weight at all: 2^(x - inf) = 0)
    lse2[g] = g < G && l[g] != 0.f ? m[g] + log2f(l[g]) : -NEG_INF;
  for (int i = i0 + static_cast<int>(threadIdx.x); i < i1; i += MASS_BATCH * NW * 32) {
    int j[MASS_BATCH];
    float old[MASS_BATCH], sum[MASS_BATCH];
#pragma unroll
    for (int b = 0; b < MASS_BATCH; ++b) {
      const int ib = i + b * NW * 32;
      j[b] = ib < i1 ? row_at(ib) : -1;
      old[b] = j[b] >= 0 ? mass[j[b]] : 0.f;
      sum[b] = 0.f;
    }
#pragma unroll
    for (int g = 0; g < MAX_GROUP; ++g) {
      if (g >= G) break;
#pragma unroll
      for (int b = 0; b < MASS_BATCH; ++b)
        if (j[b] >= 0) sum[b] += fast_exp2(logits[static_cast<int64_t>(j[b]) * G + g] - lse2[g]);
    }
#pragma unroll
    for (int b = 0; b < MASS_BATCH; ++b)
      if (j[b] >= 0) mass[j[b]] = old[b] + sum[b];
  }
}

// A cluster's runs joined (p.n_split CTAs of NW * 32 threads): tot [group][D] and
// ml [group] are each run's sums in its shared memory. This CTA's share of the
// heads' elements is written, and the masses of its own rows: row_at(i), i in
// [i0, i1), or -1.
template <typename T, int D, bool CHUNK, class RowAt>
__device__ __forceinline__ void join_cluster(const AttnParams& p, const Run& r, int ls, int split, const float* tot,
                                             const float2* ml, int i0, int i1, RowAt row_at) {
  __shared__ float s_m[MAX_GROUP], s_l[MAX_GROUP], s_a[MAX_CLUSTER][MAX_GROUP];
  const int t = threadIdx.x, G = p.group, ns = p.n_split;
  cluster_sync(ns);
  for (int g = t >> 5; g < G; g += NW) {
    // a lane per run
    const int u = t & 31;
    const float2 x = u < ns ? cluster_ld2(ml + g, u, ns) : make_float2(NEG_INF, 0.f);
    float m = x.x, l = x.y;
    const bool skip = __any_sync(FULL_MASK, l < 0.f);
#pragma unroll
    for (int k = 8; k >= 1; k >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL_MASK, m, k));
    m = m == NEG_INF ? 0.f : m;
    const float a = fast_exp2(x.x - m);
    l *= a;
#pragma unroll
    for (int k = 8; k >= 1; k >>= 1) l += __shfl_xor_sync(FULL_MASK, l, k);
    if (u < ns) s_a[u][g] = a;
    if (u == 0) {
      s_m[g] = m;
      s_l[g] = skip ? -1.f : l;
    }
  }
  __syncthreads();
  bool skip = false;
  for (int g = 0; g < G; ++g) skip |= s_l[g] < 0.f;
  if (!skip) {
    for (int i = split * NW * 32 + t; i < G * D; i += ns * NW * 32) {
      const int g = i / D, e = i % D;
      float o = 0.f;
      for (int u = 0; u < ns; ++u) o = fmaf(cluster_ld(tot + i, u, ns), s_a[u][g], o);
      store_out<T, D, CHUNK>(p, r, g, e, o, s_l[g]);
      if (e == 0) store_lse<CHUNK>(p, r, g, s_m[g], s_l[g]);
    }
    if (p.mass) {
      add_masses(p, r, ls, s_m, s_l, i0, i1, row_at);
    }
  }
  cluster_sync(ns);  // a CTA's shared memory stays until the others have read it
}

// The tiles that hold visible rows of a slice, [0, ta) and [tb, tn), and a run's
// share of them: numbers u0 .. u1 - 1 of the list.
template <typename T, int D>
struct Tiles {
  int ta, tb, u0, u1;
  int64_t base;         // of the slice's rows, and its table (kept: they take divisions)
  const int32_t* trow;
  __device__ __forceinline__ Tiles(const AttnParams& p, const Run& r, int split) {
    base = p.rows.slice_base(r.s);
    trow = p.rows.seq_table(r.s);
    constexpr int TK = TileGeo<T, D>::TK;
    const int tn = (r.n + TK - 1) / TK;
    ta = (r.vis.s1 + TK - 1) / TK;
    tb = max(ta, r.vis.w0 / TK);
    const int64_t tiles = ta + tn - tb;
    u0 = static_cast<int>(tiles * split / p.n_split);
    u1 = static_cast<int>(tiles * (split + 1) / p.n_split);
  }
  __device__ __forceinline__ int row(int u) const { return (u < ta ? u : u - ta + tb) * TileGeo<T, D>::TK; }
};

// Copies of tile u of a slice's list to `dst` (K, then V) by a warp.
template <typename T, int D, bool PAGED>
__device__ __forceinline__ void fetch_tile(const AttnParams& p, const Run& r, const Tiles<T, D>& tl, int u, uint32_t dst, int lane,
                                           bool& blocks_ok) {
  using G = TileGeo<T, D>;
  const int crow = lane / G::CH, cch = lane % G::CH, r0 = tl.row(u);
#pragma unroll
  for (int s = 0; s < G::TK / G::RUN; ++s) {
    const int rs = r0 + G::RUN * s;
    int64_t off;
    bool in = rs < r.n;
    if (PAGED) {
      int blk = 0;
      if (in) {
        blk = __ldg(tl.trow + (rs >> p.rows.block_shift));
        if (blk < 0 || blk >= p.rows.num_blocks) {
          // rows that nobody sees may have no block any more
          if (rs < r.vis.s1 || rs + G::RUN - 1 >= r.vis.w0) blocks_ok = false;
          blk = 0;
          in = false;
        }
      }
      off = tl.base + blk * p.rows.block_bytes + static_cast<int64_t>(rs & (p.rows.block_size - 1)) * G::ROW;
    } else {
      off = tl.base + static_cast<int64_t>(rs) * G::ROW;
    }
#pragma unroll
    for (int i = 0; i < G::RUN / G::RPI; ++i) {
      const int rr = i * G::RPI + crow, j = rs + rr;
      const bool live = in && j < r.n && (j < r.vis.s1 || j >= r.vis.w0);
      const int64_t o = live ? off + rr * G::ROW + cch * 16 : 0;
      const uint32_t d = (G::RUN * s + rr) * G::ROW + ((cch ^ (rr & 7)) << 4);
      cp_async16(dst + d, static_cast<const char*>(p.k) + o, live);
      cp_async16(dst + G::TILE + d, static_cast<const char*>(p.v) + o, live);
    }
  }
}

// The warps' sums of a run in shared memory, [NW][8 heads][HS], and past them the run's.
template <int D>
struct RunSums {
  static constexpr int HS = D + 4;  // floats between heads: the four lt of a store hit different banks
};
// The end of a run: its sums over the warps (so; m and l in sm_m, sm_l), then joined in the cluster or
// left for the join. bad: a block (or copy) that a visible row needs is missing.
template <class Tag, int D, bool CHUNK>
__device__ __forceinline__ void finish_run(const AttnParams& p, const Run& r, const Tiles<Tag, D>& tl, int ls, int split, int64_t pi, bool bad,
                                           float* so, const float (&sm_m)[NW][8], const float (&sm_l)[NW][8], float2* run_ml) {
  constexpr int HS = RunSums<D>::HS;
  const int t = threadIdx.x;
  __syncthreads();
  if (bad && t == 0) set_status(p.dev_status, TRI_DEV_BAD_BLOCK);
  float* tot = so + NW * 8 * HS;
  for (int i = t; i < p.group * D; i += NW * 32) {
    const int g = i / D, e = i % D;
    float m = NEG_INF;
#pragma unroll
    for (int k = 0; k < NW; ++k) m = fmaxf(m, sm_m[k][g]);
    const float mu = m == NEG_INF ? 0.f : m;
    float l = 0.f, acc = 0.f;
#pragma unroll
    for (int k = 0; k < NW; ++k) {
      const float a = fast_exp2(sm_m[k][g] - mu);
      l = fmaf(sm_l[k][g], a, l);
      acc = fmaf(so[(k * 8 + g) * HS + e], a, acc);
    }
    if (bad) l = -1.f;
    if (p.join) {
      tot[i] = acc;
      if (e == 0) run_ml[g] = make_float2(m, l);
    } else {
      p.part_o[(pi + g) * D + e] = acc;
      if (e == 0) p.part_ml[pi + g] = make_float2(m, l);
    }
  }
  constexpr int TK = TileGeo<Tag, D>::TK;
  if (p.join)
    join_cluster<__nv_bfloat16, D, CHUNK>(p, r, ls, split, tot, run_ml, tl.u0 * TK, tl.u1 * TK, [&](int i) {
      const int j = tl.row(i / TK) + i % TK;
      return j < r.n && (j < r.vis.s1 || j >= r.vis.w0) ? j : -1;
    });
}

template <int D, bool PAGED>
__global__ void __launch_bounds__(NW * 32) decode_tiles_kernel(const __grid_constant__ AttnParams p) {
  using T = __nv_bfloat16;
  using G = TileGeo<T, D>;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ float sm_m[NW][8], sm_l[NW][8];
  __shared__ float2 run_ml[MAX_GROUP];
  const int ls = blockIdx.x / p.n_split, split = blockIdx.x % p.n_split;
  const int t = threadIdx.x, w = t >> 5, lane = t & 31, lg = lane >> 2, lt = lane & 3;
  const int64_t pi = static_cast<int64_t>(blockIdx.x) * p.group;
  pdl_launch();
  Run r;
  if (!slice_run(p, ls, r)) {
    if (!p.join && t < p.group) p.part_ml[pi + t] = make_float2(NEG_INF, -1.f);
    return;  // (every run of the slice does)
  }
  const Tiles<T, D> tl(p, r, split);

  // the heads' B fragments
  uint32_t qf[D / 16][2];
  {
    const uint32_t* q = reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(p.q) + r.seq * p.q_seq +
                                                          (static_cast<int64_t>(r.h) * p.group + lg) * D);
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      qf[ks][0] = lg < p.group ? __ldg(q + ks * 8 + lt) : 0u;
      qf[ks][1] = lg < p.group ? __ldg(q + ks * 8 + lt + 4) : 0u;
    }
  }

  const uint32_t ring = smem_addr(smem) + w * G::WARP_RING;
  bool blocks_ok = true;
  auto fetch = [&](int u, int st) { fetch_tile<T, D, PAGED>(p, r, tl, u, ring + st * 2 * G::TILE, lane, blocks_ok); };

  float o[D / 16][4];
#pragma unroll
  for (int i = 0; i < D / 16; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c) o[i][c] = 0.f;
  float m0 = NEG_INF, m1 = NEG_INF, l0 = 0.f, l1 = 0.f;  // heads 2 lt, 2 lt + 1
  const float sl = p.scale * LOG2E;
  float* logits = p.logits ? p.logits + static_cast<int64_t>(ls) * p.n_cap * p.group : nullptr;

#pragma unroll
  for (int i = 0; i < G::NST - 1; ++i) {
    if (tl.u0 + w + i * NW < tl.u1) fetch(tl.u0 + w + i * NW, i);
    cp_async_commit();
  }
  int st = 0;
  for (int u = tl.u0 + w; u < tl.u1; u += NW) {
    {
      const int nx = u + (G::NST - 1) * NW, ns = st == 0 ? G::NST - 1 : st - 1;
      if (nx < tl.u1) fetch(nx, ns);
      cp_async_commit();
    }
    cp_async_wait<G::NST - 1>();
    __syncwarp();
    const int r0 = tl.row(u);
    const bool inner = r0 + G::TK <= r.n && (r0 >= r.vis.w0 || r0 + G::TK <= r.vis.s1);
    const uint32_t tk = ring + st * 2 * G::TILE, tv = tk + G::TILE;
#pragma unroll
    for (int s = 0; s < G::TK / 16; ++s) {
      float x[4] = {0.f, 0.f, 0.f, 0.f};
      {
        const int row = 16 * s + (lane & 15);
        const uint32_t a = tk + row * G::ROW;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          uint32_t kf[4];
          ldsm4(a + (((2 * ks + (lane >> 4)) ^ (row & 7)) << 4), kf);
          mma16816(x, kf, qf[ks][0], qf[ks][1]);
        }
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) x[c] *= sl;
      const int ja = r0 + 16 * s + lg, jb = ja + 8;
      if (!inner) {
        if (!(ja < r.n && (ja < r.vis.s1 || ja >= r.vis.w0))) x[0] = x[1] = NEG_INF;
        if (!(jb < r.n && (jb < r.vis.s1 || jb >= r.vis.w0))) x[2] = x[3] = NEG_INF;
      }
      if (logits) {  // (rows out of sight: their entries are not read)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int j = c < 2 ? ja : jb, g = 2 * lt + (c & 1);
          if (g < p.group && j < r.n) logits[static_cast<int64_t>(j) * p.group + g] = x[c];
        }
      }
      float mx0 = fmaxf(x[0], x[2]), mx1 = fmaxf(x[1], x[3]);
#pragma unroll
      for (int k = 4; k <= 16; k <<= 1) {
        mx0 = fmaxf(mx0, __shfl_xor_sync(FULL_MASK, mx0, k));
        mx1 = fmaxf(mx1, __shfl_xor_sync(FULL_MASK, mx1, k));
      }
      if (__any_sync(FULL_MASK, mx0 > m0 || mx1 > m1)) {
        const float n0 = fmaxf(m0, mx0), n1 = fmaxf(m1, mx1);
        const float a0 = n0 == NEG_INF ? 1.f : fast_exp2(m0 - n0), a1 = n1 == NEG_INF ? 1.f : fast_exp2(m1 - n1);
        m0 = n0;
        m1 = n1;
        l0 *= a0;
        l1 *= a1;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          o[i][0] *= a0;
          o[i][1] *= a1;
          o[i][2] *= a0;
          o[i][3] *= a1;
        }
      }
      const float z0 = m0 == NEG_INF ? 0.f : m0, z1 = m1 == NEG_INF ? 0.f : m1;
      const float e[4] = {fast_exp2(x[0] - z0), fast_exp2(x[1] - z1), fast_exp2(x[2] - z0), fast_exp2(x[3] - z1)};
      l0 += e[0] + e[2];
      l1 += e[1] + e[3];
      const uint32_t ha = pack_bf16(e[0], e[1]), hb = pack_bf16(e[2], e[3]);
      const uint32_t la = pack_bf16(e[0] - bf16_lo(ha), e[1] - bf16_hi(ha)), lb = pack_bf16(e[2] - bf16_lo(hb), e[3] - bf16_hi(hb));
      const uint32_t b0 = transpose8(ha), b1 = transpose8(hb), c0 = transpose8(la), c1 = transpose8(lb);
      const int row = 16 * s + (lane & 7) + ((lane >> 4) << 3);
      const uint32_t a = tv + row * G::ROW;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        uint32_t vf[4];
        ldsm4_t(a + (((2 * i + ((lane >> 3) & 1)) ^ (row & 7)) << 4), vf);
        mma16816(o[i], vf, b0, b1);
        mma16816(o[i], vf, c0, c1);
      }
    }
    __syncwarp();  // the stage may be refilled
    st = st + 1 == G::NST ? 0 : st + 1;
  }
  cp_async_wait<0>();
#pragma unroll
  for (int k = 4; k <= 16; k <<= 1) {
    l0 += __shfl_xor_sync(FULL_MASK, l0, k);
    l1 += __shfl_xor_sync(FULL_MASK, l1, k);
  }
  if (lg == 0) {
    sm_m[w][2 * lt] = m0;
    sm_m[w][2 * lt + 1] = m1;
    sm_l[w][2 * lt] = l0;
    sm_l[w][2 * lt + 1] = l1;
  }
  // every ring is idle: the warps' vector sums go there
  const bool bad = __syncthreads_or(PAGED && !blocks_ok);
  float* so = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int i = 0; i < D / 16; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c) so[(w * 8 + 2 * lt + (c & 1)) * RunSums<D>::HS + 16 * i + lg + (c >> 1) * 8] = o[i][c];
  finish_run<T, D, false>(p, r, tl, ls, split, pi, PAGED && bad, so, sm_m, sm_l, run_ml);
}

}  // namespace
}  // namespace tri

#include "attn_decode_q4.cuh"

namespace tri {
namespace {

// ---------------------------------------------------------------------------
// fp32 rows
// ---------------------------------------------------------------------------
constexpr int DT = NW * 32;  // threads per CTA
constexpr int LPR = 8;    // lanes per row
constexpr int GROUPS = DT / LPR;

template <int D, int GP, bool PAGED>
__global__ void __launch_bounds__(DT) decode_rows_kernel(const __grid_constant__ AttnParams p) {
  using T = float;
  using Geo = TileGeo<T, D>;
  constexpr int E = 4;              // elements per 16-byte chunk
  constexpr int C = D / (E * LPR);  // chunks per lane
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ float sq[GP][D];
  __shared__ float sm_m[GROUPS][GP], sm_l[GROUPS][GP];
  __shared__ float2 run_ml[GP];
  const int ls = blockIdx.x / p.n_split, split = blockIdx.x % p.n_split, t = threadIdx.x, G = p.group;
  const int w = t >> 5, lane = t & 31;
  pdl_launch();
  Run r;
  const int64_t pi = static_cast<int64_t>(blockIdx.x) * G;
  if (!slice_run(p, ls, r)) {
    if (!p.join && t < G) p.part_ml[pi + t] = make_float2(NEG_INF, -1.f);
    return;  // (every run of the slice does)
  }
  const Tiles<T, D> tl(p, r, split);
  const uint32_t ring = smem_addr(smem) + w * Geo::WARP_RING;
  const unsigned char* ring_p = smem + w * Geo::WARP_RING;
  bool ok = true;
  auto fetch = [&](int u, int st) { fetch_tile<T, D, PAGED>(p, r, tl, u, ring + st * 2 * Geo::TILE, lane, ok); };
#pragma unroll
  for (int i = 0; i < Geo::NST - 1; ++i) {
    if (tl.u0 + w + i * NW < tl.u1) fetch(tl.u0 + w + i * NW, i);
    cp_async_commit();
  }
  const float* q = static_cast<const float*>(p.q) + r.seq * p.q_seq + static_cast<int64_t>(r.h) * G * D;
  for (int i = t; i < GP * D; i += DT) {
    const int g = i / D;
    sq[g][i % D] = g < G ? q[i] * (p.scale * LOG2E) : 0.f;
  }
  __syncthreads();
  const int rg = t / LPR, lane8 = t % LPR;
  // up to four heads' queries stay in registers (with more, they and o do not fit)
  constexpr bool Q_REGS = GP <= 4;
  float4 qr[Q_REGS ? GP : 1][C];
  if constexpr (Q_REGS) {
#pragma unroll
    for (int g = 0; g < GP; ++g)
#pragma unroll
      for (int c = 0; c < C; ++c) qr[g][c] = *reinterpret_cast<const float4*>(&sq[g][(lane8 + LPR * c) * E]);
  }
  float m[GP], l[GP], o[GP][C * E];
#pragma unroll
  for (int g = 0; g < GP; ++g) {
    m[g] = NEG_INF;
    l[g] = 0.f;
#pragma unroll
    for (int e = 0; e < C * E; ++e) o[g][e] = 0.f;
  }
  float* logits = p.logits ? p.logits + static_cast<int64_t>(ls) * p.n_cap * G : nullptr;
  int st = 0;
  for (int u = tl.u0 + w; u < tl.u1; u += NW) {
    {
      const int nx = u + (Geo::NST - 1) * NW, ns = st == 0 ? Geo::NST - 1 : st - 1;
      if (nx < tl.u1) fetch(nx, ns);
      cp_async_commit();
    }
    cp_async_wait<Geo::NST - 1>();
    __syncwarp();
    const int r0 = tl.row(u);
#pragma unroll 1
    for (int s = 0; s < Geo::TK; s += 32 / LPR) {
      const int row = s + lane / LPR, j = r0 + row;
      const bool live = j < r.n && (j < r.vis.s1 || j >= r.vis.w0);
      const unsigned char* kp = ring_p + st * 2 * Geo::TILE + row * Geo::ROW;
      float x[GP];
#pragma unroll
      for (int g = 0; g < GP; ++g) x[g] = 0.f;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const float4 kx = *reinterpret_cast<const float4*>(kp + (((lane8 + LPR * c) ^ (row & 7)) << 4));
#pragma unroll
        for (int g = 0; g < GP; ++g) {
          const float4 qx = Q_REGS ? qr[Q_REGS ? g : 0][c] : *reinterpret_cast<const float4*>(&sq[g][(lane8 + LPR * c) * E]);
          x[g] = fmaf(qx.x, kx.x, x[g]);
          x[g] = fmaf(qx.y, kx.y, x[g]);
          x[g] = fmaf(qx.z, kx.z, x[g]);
          x[g] = fmaf(qx.w, kx.w, x[g]);
        }
      }
      float wgt[GP];
#pragma unroll
      for (int g = 0; g < GP; ++g) {
#pragma unroll
        for (int k = LPR / 2; k >= 1; k >>= 1) x[g] += __shfl_xor_sync(FULL_MASK, x[g], k);
        if (!live) x[g] = NEG_INF;
        if (logits && live && lane8 == g % LPR && g < G) logits[static_cast<int64_t>(j) * G + g] = x[g];
        if (x[g] > m[g]) {  // (the 8 lanes of a row agree)
          const float a = fast_exp2(m[g] - x[g]);
          m[g] = x[g];
          l[g] *= a;
#pragma unroll
          for (int e = 0; e < C * E; ++e) o[g][e] *= a;
        }
        wgt[g] = fast_exp2(x[g] - (m[g] == NEG_INF ? 0.f : m[g]));
        l[g] += wgt[g];
      }
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const float4 vx = *reinterpret_cast<const float4*>(kp + Geo::TILE + (((lane8 + LPR * c) ^ (row & 7)) << 4));
#pragma unroll
        for (int g = 0; g < GP; ++g) {
          o[g][c * E] = fmaf(wgt[g], vx.x, o[g][c * E]);
          o[g][c * E + 1] = fmaf(wgt[g], vx.y, o[g][c * E + 1]);
          o[g][c * E + 2] = fmaf(wgt[g], vx.z, o[g][c * E + 2]);
          o[g][c * E + 3] = fmaf(wgt[g], vx.w, o[g][c * E + 3]);
        }
      }
    }
    __syncwarp();  // the stage may be refilled
    st = st + 1 == Geo::NST ? 0 : st + 1;
  }
  cp_async_wait<0>();
  const bool bad = __syncthreads_or(PAGED && !ok);  // every ring is idle: the row groups' sums go there
  float(*so)[D] = reinterpret_cast<float(*)[D]>(smem);
  float* tot = reinterpret_cast<float*>(smem) + GROUPS * D;
  if (PAGED && bad && t == 0) set_status(p.dev_status, TRI_DEV_BAD_BLOCK);
  if (lane8 == 0) {
#pragma unroll
    for (int g = 0; g < GP; ++g) {
      sm_m[rg][g] = m[g];
      sm_l[rg][g] = l[g];
    }
  }
#pragma unroll
  for (int g = 0; g < GP; ++g) {
    if (g >= G) break;
    __syncthreads();
    float mx = NEG_INF;
    for (int u = 0; u < GROUPS; ++u) mx = fmaxf(mx, sm_m[u][g]);
    const float mu = mx == NEG_INF ? 0.f : mx;
    const float a = fast_exp2(m[g] - mu);
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int e = 0; e < E; ++e) so[rg][(lane8 + LPR * c) * E + e] = o[g][c * E + e] * a;
    __syncthreads();
    for (int e = t; e < D; e += DT) {
      float sum = 0.f;
      for (int u = 0; u < GROUPS; ++u) sum += so[u][e];
      if (p.join) tot[g * D + e] = sum;
      else p.part_o[(pi + g) * D + e] = sum;
    }
    if (t == 0) {
      float sum = 0.f;
      for (int u = 0; u < GROUPS; ++u) sum = fmaf(sm_l[u][g], fast_exp2(sm_m[u][g] - mu), sum);
      const float2 x = make_float2(mx, PAGED && bad ? -1.f : sum);
      if (p.join) run_ml[g] = x;
      else p.part_ml[pi + g] = x;
    }
  }
  if (p.join)
    join_cluster<float, D, false>(p, r, ls, split, tot, run_ml, tl.u0 * Geo::TK, tl.u1 * Geo::TK, [&](int i) {
      const int j = tl.row(i / Geo::TK) + i % Geo::TK;
      return j < r.n && (j < r.vis.s1 || j >= r.vis.w0) ? j : -1;
    });
}

// ---------------------------------------------------------------------------
// join, and masses: CTA (slice, c) of `chunks` joins head c, and with masses
// takes visible rows [c, c + 1) * JROWS: mass[j] += sum over the heads of
// 2^(x_j - m) / l.
// ---------------------------------------------------------------------------
constexpr int JT = NW * 32;
constexpr int JROWS = 1024;
constexpr int MAX_SPLIT = 128;

template <typename T, int D, bool CHUNK>
__global__ void __launch_bounds__(JT) decode_join_kernel(const __grid_constant__ AttnParams p, int chunks) {
  __shared__ float s_m[MAX_GROUP], s_l[MAX_GROUP];
  __shared__ int skip;
  const int ls = blockIdx.x / chunks, c = blockIdx.x % chunks, t = threadIdx.x, G = p.group;
  if (t == 0) skip = 0;
  pdl_wait();
  Run r;
  if (!slice_run<CHUNK>(p, ls, r)) return;
  __syncthreads();
  // (m, l) of the heads: a warp per head, lanes over the runs
  const float2* ml = p.part_ml + static_cast<int64_t>(ls) * p.n_split * G;
  for (int g = t >> 5; g < G; g += JT / 32) {
    if (!p.mass && g != c) continue;
    float m = NEG_INF, l = 0.f;
    for (int i = t & 31; i < p.n_split; i += 32) {
      const float2 x = ml[i * G + g];
      if (x.y < 0.f) skip = 1;
      m = fmaxf(m, x.x);
    }
#pragma unroll
    for (int k = 16; k >= 1; k >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL_MASK, m, k));
    const float mu = m == NEG_INF ? 0.f : m;
    for (int i = t & 31; i < p.n_split; i += 32) {
      const float2 x = ml[i * G + g];
      l = fmaf(x.y, fast_exp2(x.x - mu), l);
    }
#pragma unroll
    for (int k = 16; k >= 1; k >>= 1) l += __shfl_xor_sync(FULL_MASK, l, k);
    if ((t & 31) == 0) {
      s_m[g] = mu;
      s_l[g] = l;
    }
  }
  __syncthreads();
  if (skip) return;
  if (c < G) {
    const float* po = p.part_o + (static_cast<int64_t>(ls) * p.n_split * G + c) * D;
    for (int e = t; e < D; e += JT) {
      float o = 0.f;
#pragma unroll 4
      for (int i = 0; i < p.n_split; ++i) o = fmaf(po[static_cast<int64_t>(i) * G * D + e], fast_exp2(ml[i * G + c].x - s_m[c]), o);
      store_out<T, D, CHUNK>(p, r, c, e, o, s_l[c]);
    }
    if (t == 0) store_lse<CHUNK>(p, r, c, s_m[c], s_l[c]);
  }
  if (!p.mass) return;
  add_masses(p, r, ls, s_m, s_l, c * JROWS, min(r.count, (c + 1) * JROWS),
             [&](int i) { return i < r.vis.s1 ? i : i - r.vis.s1 + r.vis.w0; });
}

template <typename T, int D, bool CHUNK = false>
cudaError_t launch_join(const AttnParams& p, int max_rows, cudaStream_t st) {
  const int chunks = p.mass ? max(p.group, (max_rows + JROWS - 1) / JROWS) : p.group;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(p.n_seq * p.n_kv_heads * max(p.passes, 1) * chunks));
  cfg.blockDim = dim3(JT);
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, decode_join_kernel<T, D, CHUNK>, p, chunks);
  if (e == cudaSuccess) note_launch();
  return e;
}

// The runs, as clusters of a slice's when they join there.
template <class Kernel>
cudaError_t launch_runs(Kernel kern, size_t smem, const AttnParams& p, cudaStream_t st) {
  cudaError_t e;
  if (smem > 46 * 1024) {  // (48 KB, static shared memory included, need no asking for)
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  const unsigned ctas = static_cast<unsigned>(p.n_seq * p.n_kv_heads * max(p.passes, 1) * p.n_split);
  if (p.join && p.n_split > 1) {
    if (p.n_split > 8) {
      e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(NW * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = static_cast<unsigned>(p.n_split);
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kern, p);
  } else {
    kern<<<ctas, NW * 32, smem, st>>>(p);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess) note_launch();
  return e;
}

template <int D>
cudaError_t launch_bf16(const AttnParams& p, int max_rows, cudaStream_t st) {
  const cudaError_t e = launch_runs(p.rows.table ? decode_tiles_kernel<D, true> : decode_tiles_kernel<D, false>,
                                    TileGeo<__nv_bfloat16, D>::SMEM, p, st);
  return e != cudaSuccess || p.join ? e : launch_join<__nv_bfloat16, D>(p, max_rows, st);
}

template <int D>
cudaError_t launch_q4(const AttnParams& p, int max_rows, cudaStream_t st) {
  using G = TileGeo<Q4Tag, D>;
  const bool whole = p.rows.block_size >= G::TK;
  auto kern = p.token_heads ? (!p.rows.table ? decode_q4_kernel<D, SLICES, true>
                               : whole       ? decode_q4_kernel<D, WHOLE_TILES, true>
                                             : decode_q4_kernel<D, SMALL_BLOCKS, true>)
                            : (!p.rows.table ? decode_q4_kernel<D, SLICES, false>
                               : whole       ? decode_q4_kernel<D, WHOLE_TILES, false>
                                             : decode_q4_kernel<D, SMALL_BLOCKS, false>);
  const cudaError_t e = launch_runs(kern, G::SMEM, p, st);
  if (e != cudaSuccess || p.join) return e;
  return p.token_heads ? launch_join<__nv_bfloat16, D, true>(p, max_rows, st) : launch_join<__nv_bfloat16, D>(p, max_rows, st);
}

template <int D, int GP>
cudaError_t launch_fp32_group(const AttnParams& p, cudaStream_t st) {
  return launch_runs(p.rows.table ? decode_rows_kernel<D, GP, true> : decode_rows_kernel<D, GP, false>, TileGeo<float, D>::SMEM, p, st);
}

template <int D>
cudaError_t launch_fp32(const AttnParams& p, int max_rows, cudaStream_t st) {
  const cudaError_t e = p.group == 1 ? launch_fp32_group<D, 1>(p, st) : p.group == 2 ? launch_fp32_group<D, 2>(p, st)
                      : p.group <= 4 ? launch_fp32_group<D, 4>(p, st) : launch_fp32_group<D, 8>(p, st);
  return e != cudaSuccess || p.join ? e : launch_join<float, D>(p, max_rows, st);
}

}  // namespace

int attn_decode_max_splits(int n_slices, int max_rows) {
  const int fill = max(MAX_CLUSTER, 608 / n_slices), most = (max_rows + 63) / 64;
  return max(1, min(min(MAX_SPLIT, fill), most));
}

// Runs per slice of a 4-bit cache, for slices of max_rows. Measured (us; back to back; c: joined in a
// cluster, k: by a second kernel; d 128, group 4, the last line d 64, group 1):
//   slices x rows   1c    2c    4c    8c    2k    4k    7k    8k    14k   19k   38k
//     8 x 2113     20.8  15.9  12.6  10.8  14.6  12.6  12.4  10.6  12.6  12.6   -
//     8 x 32768   174.8  92.7  51.7  31.2  92.7  51.7  35.1  31.2  23.1  21.2  21.0
//    32 x 8192     51.7  31.2  21.0  16.9  31.2  21.0  20.8  18.8  19.0  19.0  24.3
//   128 x 8192     55.6  43.7  41.7  45.8  43.9  41.7  42.1  41.7  45.8  50.1   -
//   128 x 32768   203.9 144.1 131.2 134.5 144.9 131.8 121.1 121.1 123.6 126.5   -
//   256 x 2048     25.5  25.5  28.0  38.6  25.5  26.9  31.7  31.7  41.9   -     -
//   512 x 2176     29.2  32.1  41.9   -    30.2  33.9  41.7   -     -     -     -
// Four CTAs fit an SM. A cluster of the largest power of two whose runs are there at once; few slices of long
// rows need more runs than a cluster holds, two CTAs per SM of them (each has its start and its sums to join);
// runs of 4096 rows and more are cut in two, so that what an SM lacks at the end is shorter; and where a
// cluster's runs would leave a fifth of the last wave empty, more runs that fill it.
static DecodePlan attn_decode_plan_q4(int n_slices, int max_rows) {
  const int64_t n = n_slices, slots = 4 * 152;
  int s = 1;
  while (2 * s <= MAX_CLUSTER && n * 2 * s <= slots && max_rows >= 64 * 2 * s) s *= 2;
  const int64_t few = min(slots / 2 / n, static_cast<int64_t>(max_rows / 384));
  if (few > s) return {static_cast<int>(min(few, static_cast<int64_t>(MAX_SPLIT))), false};
  if (max_rows / s >= 4096 && 2 * s <= attn_decode_max_splits(n_slices, max_rows)) return {2 * s, false};  // (as many as the workspace holds)
  for (int k = s; k <= 4 * s && max_rows >= 512 * k; ++k)
    if (n * k * 5 >= (n * k + slots - 1) / slots * slots * 4) return {k, k == s};
  return {s, true};
}

// Runs per slice, for slices of max_rows. Measured (us; bf16, d 128, group 4;
// c: joined in a cluster, k: by a second kernel):
//   slices x rows   1c    2c    4c    8c    16c   3k    6k    12k   19k   38k   76k
//     8 x 2113     24.6  15.2  10.1   7.9   7.9  12.5   8.8   7.6   8.2   9.7    -
//     8 x 32768   305.4 156.4  82.0  45.3  32.5 107.3  58.1  35.1  30.5  29.5  36.4
//    32 x 8192     82.4  45.6  29.2  25.4  33.0  35.2  28.0  27.6  31.7  34.0  42.7
//   128 x 8192     95.9  80.5  95.5  88.3 103.2  85.2  83.2  86.3  88.8  94.0    -
//   256 x 2048     45.4  56.2  52.2  57.2  97.9  47.7  50.6  54.1  58.3    -     -
// and fp32, group 1:
//    64 x 2048     50.2  30.6  25.2  31.8  38.0  28.8  26.9  27.6  30.7  36.5    -
//   128 x 8192    194.8 152.8 185.6 160.2 171.5 161.5 153.8 156.2 158.1 160.7    -
// A run's start and end cost a few microseconds, so the best has as few runs as
// fill the GPU once (`slots` of them) and no more: a cluster of the largest
// power of two within that. Few slices of long rows need more runs than a
// cluster holds; more slices than slots that leave the last wave part empty are
// cut into a few runs (512 slices of 2048 rows, d 64, group 1, masses: 1c 62.9,
// 3k 54.4).
DecodePlan attn_decode_plan(int n_slices, int max_rows, tri_dtype dt) {
  if (dt == TRI_Q4) return attn_decode_plan_q4(n_slices, max_rows);
  const int64_t n = n_slices, slots = 2 * 152;
  int s = 1;
  while (2 * s <= MAX_CLUSTER && n * 2 * s <= slots && max_rows >= 64 * 2 * s) s *= 2;
  if (n * s * 3 <= slots * 2 && max_rows >= 512 * s) {
    const int64_t k = min(min(slots / n, static_cast<int64_t>(max_rows / 384)), static_cast<int64_t>(MAX_SPLIT));
    if (k > s) return {static_cast<int>(k), false};
  }
  if (n > slots && max_rows >= 4 * 512) {
    constexpr int64_t WAVE = 3 * 152;
    for (int k = 1; k <= 4; ++k)
      if (n * k * 5 >= (n * k + WAVE - 1) / WAVE * WAVE * 4) return {k, k == 1};
  }
  return {s, true};
}

cudaError_t launch_attn_decode(const AttnParams& p, int max_rows, tri_dtype dt, int head_dim, cudaStream_t st) {
  if (dt == TRI_Q4) return head_dim == 64 ? launch_q4<64>(p, max_rows, st) : launch_q4<128>(p, max_rows, st);
  if (dt == TRI_BF16) return head_dim == 64 ? launch_bf16<64>(p, max_rows, st) : launch_bf16<128>(p, max_rows, st);
  return head_dim == 64 ? launch_fp32<64>(p, max_rows, st) : launch_fp32<128>(p, max_rows, st);
}

}  // namespace tri
