// attn_decode_q4.cuh -- the decode kernel over rows in 4 bits (included by
// attn_decode.cu, whose runs, joins and masses it shares).
//
// A row is codes c and per quarter j of its elements a scale s_j and a minimum m_j:
//   q . k = sum_j (s_j sum_e q_e c_e + m_j sum_e q_e),
//   sum_r p_r v_r = sum_r (p_r s_rj) c_re + sum_r p_r m_rj   (e in quarter j),
// so the products run on the codes, and scales and minima enter outside of them.
//
// Bound: 2 (d / 2 + 16) bytes a row pair, 160 instead of 512 at d 128. At the copy rate
// that is 35 elements per clock and SM, so what it takes to bring 4 bits to an
// operand decides: an fp16 whose exponent is 0 and whose low bits are c is the number
// c 2^-24 (the tensor cores take subnormals as they are), four bits higher it
// is c 2^-20. A word of eight codes is then four ANDs and one shift: pairs
// (0, 4), (1, 5) << 4, (2, 6), (3, 7) << 4, with no offset to take off again; the
// powers of two go into q and into the final scaling.
//   S = K Q^T: A = 16 rows' codes. Lane (g, t) reads 16 (d 64: 8) bytes of rows g and g + 8,
//   its elements of all four quarters (the row's order of codes is made for
//   that); per quarter one or two MMAs whose sums are scaled per row in fp32.
//   q as fp16, scaled by a power of two so that the head's largest is below 2^15: exact
//   for every element down to 2^-25 of it. Minima: one MMA against the quarters' sums of
//   q as fp16 pairs.
//   O^T += V^T P^T: A = V transposed, 16 elements of a quarter x 16 rows. Two rows' codes of
//   an element come together by a byte permute of their words, before they are
//   spread. B = p (2^k s_j) in fp16: two roundings of 2^-11 of its weight, where results are
//   rounded to 2^-8. p is up to 2^11 and 2^k s_j up to 2^5, k from the warp's largest scale so far (a
//   larger one lowers it, and the sums so far with it), so that what falls to fp16's subnormal numbers
//   and below is 2^-36 of the largest weight times the largest value (2^-11 at least, as 2^k is an
//   fp16 number too). (With k 0 and p up to 2^4, a row 14 above the others in the logit left these
//   without their codes where V's elements were about 2^-10.) For this a lane per row reads the row's
//   pairs in shared memory and puts them back as the products take them: two rows' scales, times
//   2^k, then two rows' minima. The quarter of the loads that this saves pays for it (16 x 8 x 32768
//   rows 119.8 us, without k 119.7, with the pairs left in their order 123.8).
// Each warp owns a ring of NST tiles of 32 (d 64: 64) rows, K and V, filled by 16-byte asynchronous copies
// of whole contiguous tiles (bulk copies by lanes of a warp took 20 instructions more per 16 rows
// than these); table entries are read a tile ahead. Rows out of sight are copied but not
// used: their weight and their pairs (any bits) are set to zero.
#pragma once

#include "q4_common.cuh"

namespace tri {
namespace {

struct Q4Tag {};
template <int D>
struct TileGeo<Q4Tag, D> {
  static constexpr int ROW = Q4Row<D>::BYTES;
  static constexpr int TK = D == 64 ? 64 : 32;  // (3 and 2.5 KB of K: half the loop's overhead at d 64)
  static constexpr int TILE = TK * ROW;
  static constexpr int NST = 2;
  static constexpr int WARP_RING = NST * 2 * TILE;
  static constexpr int SMEM = NW * WARP_RING;
};

__device__ __forceinline__ void mma16816h(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The first product of a sum.
__device__ __forceinline__ void mma16816h_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void cp_async16_all(uint32_t dst, const char* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_half2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));  // (the number, where one is a NaN)
  return r;
}
__device__ __forceinline__ float scale_of(uint32_t pair) { return __low2float(*reinterpret_cast<const __half2*>(&pair)); }
// A lane's words of a row of codes.
template <int N>
__device__ __forceinline__ void lds_words(uint32_t a, uint32_t (&w)[N]) {
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(a) : "memory");
  else
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(a) : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t x;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(x) : "r"(a) : "memory");
  return x;
}

__device__ __forceinline__ void sts4(uint32_t a, const uint32_t (&w)[4]) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
}

// A head's query as B fragments for the codes (see the file comment), by the four
// lanes of the head: f[mma][2], the sums of its quarters as an fp16 pair (lane t: quarter t), and
// log2 of the power of two in them.
template <int D>
__device__ __forceinline__ void query_fragments(const __nv_bfloat16* q, bool live, int t, uint32_t (&f)[D / 16][2], uint32_t& sums, int& shift) {
  float x[4][D / 16];  // [quarter][the lane's elements]
  float most = 0.f, sum[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __nv_bfloat16* at = q + j * (D / 4) + t * (D / 16);
    uint32_t w[D / 32];
#pragma unroll
    for (int k = 0; k < D / 32; ++k) w[k] = live ? __ldg(reinterpret_cast<const uint32_t*>(at) + k) : 0u;
    sum[j] = 0.f;
#pragma unroll
    for (int k = 0; k < D / 32; ++k) {
      x[j][2 * k] = bf16_lo(w[k]);
      x[j][2 * k + 1] = bf16_hi(w[k]);
      most = fmaxf(most, fmaxf(fabsf(x[j][2 * k]), fabsf(x[j][2 * k + 1])));
      sum[j] += x[j][2 * k] + x[j][2 * k + 1];
    }
  }
#pragma unroll
  for (int k = 1; k <= 2; k <<= 1) {
    most = fmaxf(most, __shfl_xor_sync(FULL_MASK, most, k));
#pragma unroll
    for (int j = 0; j < 4; ++j) sum[j] += __shfl_xor_sync(FULL_MASK, sum[j], k);
  }
  // most 2^shift in [2^14, 2^15)
  const int e = static_cast<int>(__float_as_uint(most) >> 23) - 127;
  shift = most == 0.f ? 0 : min(max(14 - e, -100), 100);
  const float up = __uint_as_float(static_cast<uint32_t>(127 + shift) << 23);
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int k = 0; k < D / 16; ++k) x[j][k] *= up;
  if constexpr (D == 128) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        f[2 * j + h][0] = pack_half(x[j][2 * h], x[j][2 * h + 4]);
        f[2 * j + h][1] = pack_half(x[j][2 * h + 1] * 0.0625f, x[j][2 * h + 5] * 0.0625f);
      }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[j][0] = pack_half(x[j][0], x[j][2]);
      f[j][1] = pack_half(x[j][1] * 0.0625f, x[j][3] * 0.0625f);
    }
  }
  const float s = (t == 0 ? sum[0] : t == 1 ? sum[1] : t == 2 ? sum[2] : sum[3]) * up * 0.03125f;
  const float hi = __half2float(__float2half_rn(s));
  sums = pack_half(hi, s - hi);
}

// BLOCKS: how the cache's rows lie. CHUNK: the columns are the heads of a few tokens, each with its own last row (the
// pass's tokens are some of the chunk's); tiles at the edge of what some token sees are masked column by column.
enum Q4Blocks { SLICES, WHOLE_TILES, SMALL_BLOCKS };  // slices; pools whose blocks hold whole tiles, or not
template <int D, Q4Blocks BLOCKS, bool CHUNK>
__global__ void __launch_bounds__(NW * 32, 4) decode_q4_kernel(const __grid_constant__ AttnParams p) {
  using G = TileGeo<Q4Tag, D>;
  constexpr bool PAGED = BLOCKS != SLICES, whole = BLOCKS != SMALL_BLOCKS;
  constexpr int NWD = Q4Row<D>::WORDS, CODES = Q4Row<D>::CODES, LANE = 4 * NWD;  // bytes of a lane's codes
  constexpr float LIFT = 11.f;  // log2 of the largest weight
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ float sm_m[NW][8], sm_l[NW][8];
  __shared__ float2 run_ml[MAX_GROUP];
  const int ls = blockIdx.x / p.n_split, split = blockIdx.x % p.n_split;
  const int t = threadIdx.x, w = t >> 5, lane = t & 31, lg = lane >> 2, lt = lane & 3;
  const int64_t pi = static_cast<int64_t>(blockIdx.x) * p.group;
  pdl_launch();
  Run r;
  if (!slice_run<CHUNK>(p, ls, r)) {
    if (!p.join && t < p.group) p.part_ml[pi + t] = make_float2(NEG_INF, -1.f);
    return;  // (every run of the slice does)
  }
  const Tiles<Q4Tag, D> tl(p, r, split);

  // The warp's ring. A tile's rows lie in one run, or in several of smaller blocks, whose table
  // entries (-1: no row there) are read a tile before the copies.
  constexpr int SUB = G::TK / 16;                       // MMAs' rows of a tile
  constexpr int CHUNKS = G::TILE / 16, PER_LANE = CHUNKS / 32;  // 16-byte chunks of one tensor's tile
  static_assert(CHUNKS % 32 == 0, "a tile in whole copies of a warp");
  const uint32_t ring = smem_addr(smem) + w * G::WARP_RING;
  bool blocks_ok = true;
  const char *kbase = static_cast<const char*>(p.k) + tl.base, *vbase = static_cast<const char*>(p.v) + tl.base;
  struct Blocks {
    int b[whole ? 1 : SUB];  // of rows 16 k on; whole tiles: of all
  };
  auto look_up = [&](int u) {
    Blocks b;
    const int r0 = tl.row(u);
#pragma unroll
    for (int k = 0; k < (whole ? 1 : SUB); ++k)
      b.b[k] = PAGED && u < tl.u1 && r0 + 16 * k < r.n ? __ldg(tl.trow + ((r0 + 16 * k) >> p.rows.block_shift)) : -1;
    return b;
  };
  auto fetch = [&](int u, int st, const Blocks& b) {
    const int r0 = tl.row(u);
    const uint32_t dst = ring + 2 * st * G::TILE + 16 * lane;
    if (r0 + G::TK <= r.n && whole && (!PAGED || (b.b[0] >= 0 && b.b[0] < p.rows.num_blocks))) {
      const int at = PAGED ? r0 & (p.rows.block_size - 1) : r0;
      const int64_t off = (PAGED ? b.b[0] * p.rows.block_bytes : 0) + static_cast<int64_t>(at) * G::ROW + 16 * lane;
#pragma unroll
      for (int i = 0; i < PER_LANE; ++i) {
        cp_async16_all(dst + 512 * i, kbase + off + 512 * i);
        cp_async16_all(dst + G::TILE + 512 * i, vbase + off + 512 * i);
      }
      return;
    }
    if (!whole) {
      // (a tile holds whole blocks, so a chunk's place in its block is the same in every tile)
      int64_t at[SUB];
      bool all = r0 + G::TK <= r.n;
#pragma unroll
      for (int k = 0; k < SUB; ++k) {
        at[k] = b.b[whole ? 0 : k] * p.rows.block_bytes;
        all &= b.b[whole ? 0 : k] >= 0 && b.b[whole ? 0 : k] < p.rows.num_blocks;
      }
      if (all) {
#pragma unroll
        for (int i = 0; i < PER_LANE; ++i) {
          const int c = lane + 32 * i, row = c / (G::ROW / 16), k = row / 16;
          int64_t off = at[0];
#pragma unroll
          for (int x = 1; x < SUB; ++x) off = k == x ? at[x] : off;
          off += (row & (p.rows.block_size - 1)) * G::ROW + 16 * (c - row * (G::ROW / 16));
          cp_async16_all(dst + 512 * i, kbase + off);
          cp_async16_all(dst + G::TILE + 512 * i, vbase + off);
        }
        return;
      }
    }
    uint32_t bad = 0;  // bit k: rows 16 k on have no block
    if (PAGED) {
#pragma unroll
      for (int k = 0; k < SUB; ++k) {
        const int blk = b.b[whole ? 0 : k], rs = r0 + 16 * k;
        if (rs >= r.n || (blk >= 0 && blk < p.rows.num_blocks)) continue;
        bad |= 1u << k;
        // rows that nobody sees may have no block any more
        if (rs < r.vis.s1 || rs + 15 >= r.vis.w0) blocks_ok = false;
      }
    }
#pragma unroll
    for (int i = 0; i < PER_LANE; ++i) {  // rows that are not there: zeros
      const int c = lane + 32 * i, row = c / (G::ROW / 16), k = row / 16, j = r0 + row;
      const bool live = j < r.n && !(bad >> k & 1);
      int64_t off;
      if (PAGED) {
        int blk = b.b[0];
#pragma unroll
        for (int x = 1; x < (whole ? 1 : SUB); ++x) blk = k == x ? b.b[x] : blk;
        off = blk * p.rows.block_bytes + static_cast<int64_t>(j & (p.rows.block_size - 1)) * G::ROW;
      } else {
        off = static_cast<int64_t>(j) * G::ROW;
      }
      off += 16 * (c - row * (G::ROW / 16));
      cp_async16(dst + 512 * i, kbase + (live ? off : 0), live);
      cp_async16(dst + G::TILE + 512 * i, vbase + (live ? off : 0), live);
    }
  };
  Blocks ahead{};
#pragma unroll
  for (int i = 0; i < G::NST - 1; ++i) {
    const int u = tl.u0 + w + i * NW;
    if (u < tl.u1) fetch(u, i, look_up(u));
    cp_async_commit();
  }
  ahead = look_up(tl.u0 + w + (G::NST - 1) * NW);

  // the heads' B fragments, and what their products are to be multiplied with (heads 2 lt, 2 lt + 1)
  uint32_t qf[D / 16][2], qsum;
  float f0, f1;
  {
    int shift;
    const int tok = CHUNK ? lg / p.token_heads : 0, heads = CHUNK ? p.token_heads : p.group;
    query_fragments<D>(static_cast<const __nv_bfloat16*>(p.q) + r.seq * p.q_seq + (CHUNK ? (r.tok0 + tok) * p.q_token : 0) +
                           (static_cast<int64_t>(r.h) * heads + lg - tok * heads) * D,
                       lg < p.group && (!CHUNK || tok < r.news), lt, qf, qsum, shift);
    const int s0 = __shfl_sync(FULL_MASK, shift, 8 * lt), s1 = __shfl_sync(FULL_MASK, shift, 8 * lt + 4);
    const float sl = p.scale * LOG2E;
    // (not 0, which an invisible row's -inf would not survive)
    f0 = fmaxf(sl * __uint_as_float(static_cast<uint32_t>(127 + 24 - s0) << 23), 0x1p-126f);
    f1 = fmaxf(sl * __uint_as_float(static_cast<uint32_t>(127 + 24 - s1) << 23), 0x1p-126f);
  }

  float o[D / 16][4], om[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < D / 16; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c) o[i][c] = 0.f;
  // heads 2 lt, 2 lt + 1: weights are 2^(x - m), m at least the largest x minus LIFT
  float m0 = NEG_INF, m1 = NEG_INF, l0 = 0.f, l1 = 0.f;
  // V's scales, and so o, are times 2^k, k <= 15 so that 2^k is an fp16 number: 2^(5 - k), which scales stay below, as fp16
  uint32_t lim = (20 - 15) << 10;
  float* logits = p.logits ? p.logits + static_cast<int64_t>(ls) * p.n_cap * p.group : nullptr;
  const uint32_t half_sel = lg >= 4 ? 0x7632 : 0x5410;
  // A tile's rows r0 .. from `tk`; all: every one of them is in sight.
  auto tile = [&](auto all, int r0, uint32_t tk) {
    constexpr bool INNER = decltype(all)::value;
    const uint32_t tv = tk + G::TILE;
    float x[SUB][4];
#pragma unroll
    for (int s = 0; s < SUB; ++s) {
      const uint32_t ra = tk + (16 * s + lg) * G::ROW, rb = ra + 8 * G::ROW;
      uint32_t wa[NWD], wb[NWD], pa[4], pb[4];
      lds_words(ra + LANE * lt, wa);
      lds_words(rb + LANE * lt, wb);
      lds_words(ra + CODES, pa);
      lds_words(rb + CODES, pb);
      {
        const uint32_t ma = lds32(ra + CODES + 4 * lt), mb = lds32(rb + CODES + 4 * lt);
        float y[4];
        mma16816h_first(y, __byte_perm(ma, ma, 0x3232), __byte_perm(mb, mb, 0x3232), 0u, 0u, qsum, 0u);
#pragma unroll
        for (int c = 0; c < 4; ++c) x[s][c] = y[c] * 0x1p-19f;
      }
#pragma unroll
      for (int k = 0; k < NWD; ++k) {
        const uint32_t a8 = wa[k] >> 8, b8 = wb[k] >> 8;
        constexpr uint32_t LO = 0x000f000fu, HI = 0x00f000f0u;
        float y[4];
        mma16816h_first(y, wa[k] & LO, wb[k] & LO, wa[k] & HI, wb[k] & HI, qf[2 * k][0], qf[2 * k][1]);
        if constexpr (D == 64) {
          const float sa = scale_of(pa[2 * k]), sb = scale_of(pb[2 * k]);
          x[s][0] = fmaf(y[0], sa, x[s][0]);
          x[s][1] = fmaf(y[1], sa, x[s][1]);
          x[s][2] = fmaf(y[2], sb, x[s][2]);
          x[s][3] = fmaf(y[3], sb, x[s][3]);
          mma16816h_first(y, a8 & LO, b8 & LO, a8 & HI, b8 & HI, qf[2 * k + 1][0], qf[2 * k + 1][1]);
        } else {
          mma16816h(y, a8 & LO, b8 & LO, a8 & HI, b8 & HI, qf[2 * k + 1][0], qf[2 * k + 1][1]);
        }
        constexpr int QS = D == 64 ? 2 : 1;
        const float sa = scale_of(pa[QS * k + QS - 1]), sb = scale_of(pb[QS * k + QS - 1]);
        x[s][0] = fmaf(y[0], sa, x[s][0]);
        x[s][1] = fmaf(y[1], sa, x[s][1]);
        x[s][2] = fmaf(y[2], sb, x[s][2]);
        x[s][3] = fmaf(y[3], sb, x[s][3]);
      }
      const int ja = r0 + 16 * s + lg, jb = ja + 8;
      if (!INNER) {
        if constexpr (CHUNK) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int j = c < 2 ? ja : jb, last = r.first + (2 * lt + (c & 1)) / p.token_heads;
            const Visible v = visible_rows(last, p.n_sink, p.window);
            if (!(j < r.n && j <= last && (j < v.s1 || j >= v.w0))) x[s][c] = NEG_INF;
          }
        } else {
          if (!(ja < r.n && (ja < r.vis.s1 || ja >= r.vis.w0))) x[s][0] = x[s][1] = NEG_INF;
          if (!(jb < r.n && (jb < r.vis.s1 || jb >= r.vis.w0))) x[s][2] = x[s][3] = NEG_INF;
        }
      }
      if (logits) {  // (rows out of sight: their entries are not read)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int j = c < 2 ? ja : jb, g = 2 * lt + (c & 1);
          if (g < p.group && j < r.n) logits[static_cast<int64_t>(j) * p.group + g] = x[s][c] * (c & 1 ? f1 : f0);
        }
      }
    }
    // V's pairs, a lane per row: zeros for rows out of sight (any bits), the scales of others times 2^k
    uint32_t pv[G::TK / 32][4], most = 0;
#pragma unroll
    for (int i = 0; i < G::TK / 32; ++i) lds_words(tv + (lane + 32 * i) * G::ROW + CODES, pv[i]);
    float mx0 = fmaxf(x[0][0], x[0][2]), mx1 = fmaxf(x[0][1], x[0][3]);
#pragma unroll
    for (int s = 1; s < SUB; ++s) {
      mx0 = fmaxf(fmaxf(mx0, x[s][0]), x[s][2]);
      mx1 = fmaxf(fmaxf(mx1, x[s][1]), x[s][3]);
    }
    // (rounded up: to the nearest, logits of 2^17 give weights of 2^(LIFT + 1/64), which times the largest scale is past fp16)
    mx0 = __fmaf_ru(mx0, f0, -LIFT);
    mx1 = __fmaf_ru(mx1, f1, -LIFT);
#pragma unroll
    for (int i = 0; i < G::TK / 32; ++i) {
      const int j = r0 + lane + 32 * i;
      if (!INNER && !(j < r.n && (j < r.vis.s1 || j >= r.vis.w0))) pv[i][0] = pv[i][1] = pv[i][2] = pv[i][3] = 0u;
      most = max_half2(most, max_half2(max_half2(pv[i][0], pv[i][1]), max_half2(pv[i][2], pv[i][3])));
    }
    most &= 0xffffu;
    if (__any_sync(FULL_MASK, mx0 > m0 || mx1 > m1 || most >= lim)) {
#pragma unroll
      for (int k = 4; k <= 16; k <<= 1) {
        mx0 = fmaxf(mx0, __shfl_xor_sync(FULL_MASK, mx0, k));
        mx1 = fmaxf(mx1, __shfl_xor_sync(FULL_MASK, mx1, k));
      }
      // (a scale that is new is 2^-10 at least; infinite ones stay as they are)
      const uint32_t next = max(lim, (min(__reduce_max_sync(FULL_MASK, most) >> 10, 30u) + 1) << 10);
      const float n0 = fmaxf(m0, mx0), n1 = fmaxf(m1, mx1), ak = __uint_as_float((127 + (lim >> 10) - (next >> 10)) << 23);
      float a0 = n0 == NEG_INF ? 1.f : fast_exp2(m0 - n0), a1 = n1 == NEG_INF ? 1.f : fast_exp2(m1 - n1);
      m0 = n0;
      m1 = n1;
      lim = next;
      l0 *= a0;
      l1 *= a1;
      om[0] *= a0;
      om[1] *= a1;
      a0 *= ak;
      a1 *= ak;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        o[i][0] *= a0;
        o[i][1] *= a1;
        o[i][2] *= a0;
        o[i][3] *= a1;
      }
    }
    // two rows' words of scales go to the pairs of the even row, those of minima to the odd one's
    const bool odd = lane & 1;
    const uint32_t up = odd ? 0x3c003c00u : __byte_perm((35u << 10) - lim, 0, 0x1010);  // 2^k, minima as they are
#pragma unroll
    for (int i = 0; i < G::TK / 32; ++i) {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t own = __byte_perm(pv[i][2 * k], pv[i][2 * k + 1], odd ? 0x7632 : 0x5410);
        const uint32_t other = __shfl_xor_sync(FULL_MASK, __byte_perm(pv[i][2 * k], pv[i][2 * k + 1], odd ? 0x5410 : 0x7632), 1);
        w[2 * k] = mul_half2(__byte_perm(own, other, odd ? 0x1054 : 0x5410), up);
        w[2 * k + 1] = mul_half2(__byte_perm(own, other, odd ? 0x3276 : 0x7632), up);
      }
      sts4(tv + (lane + 32 * i) * G::ROW + CODES, w);
    }
    __syncwarp();  // (the pairs)
    const float z0 = !INNER && m0 == NEG_INF ? 0.f : m0, z1 = !INNER && m1 == NEG_INF ? 0.f : m1;
#pragma unroll
    for (int s = 0; s < SUB; ++s) {
      const float e[4] = {fast_exp2(fmaf(x[s][0], f0, -z0)), fast_exp2(fmaf(x[s][1], f1, -z1)), fast_exp2(fmaf(x[s][2], f0, -z0)),
                          fast_exp2(fmaf(x[s][3], f1, -z1))};
      l0 += e[0] + e[2];
      l1 += e[1] + e[3];
      const uint32_t p01 = transpose8(pack_half(e[0], e[1])), p89 = transpose8(pack_half(e[2], e[3]));  // rows 2 lt, + 1, + 8, + 9; head lg
      uint32_t vw[4][NWD], b0[4], b1[4];
      const uint32_t ra = tv + (16 * s + 2 * lt) * G::ROW;
#pragma unroll
      for (int k = 0; k < 4; ++k) lds_words(ra + ((k & 1) + 8 * (k >> 1)) * G::ROW + LANE * (lg & 3), vw[k]);
      lds_words(ra + CODES, b0);
      lds_words(ra + 8 * G::ROW + CODES, b1);
      mma16816h(om, lds32(ra + G::ROW + CODES + 4 * (lg & 3)), 0u, lds32(ra + 9 * G::ROW + CODES + 4 * (lg & 3)), 0u, p01, p89);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        b0[j] = mul_half2(p01, b0[j]);
        b1[j] = mul_half2(p89, b1[j]);
      }
#pragma unroll
      for (int k = 0; k < NWD; ++k) {
        const uint32_t y01 = __byte_perm(vw[0][k], vw[1][k], half_sel), y89 = __byte_perm(vw[2][k], vw[3][k], half_sel);
        const uint32_t z01 = y01 >> 8, z89 = y89 >> 8;
        constexpr uint32_t LO = 0x000f000fu, HI = 0x00f000f0u;
        const int ja = D == 64 ? 2 * k : k, jb = D == 64 ? 2 * k + 1 : k;
        mma16816h(o[2 * k], y01 & LO, y01 & HI, y89 & LO, y89 & HI, b0[ja], b1[ja]);
        mma16816h(o[2 * k + 1], z01 & LO, z01 & HI, z89 & LO, z89 & HI, b0[jb], b1[jb]);
      }
    }
  };
  // rows below all_s1, and from all_w0 up to all_end, are in every column's sight
  int all_end = r.n, all_w0 = r.vis.w0, all_s1 = r.vis.s1;
  if constexpr (CHUNK) {
    all_end = max(r.first + 1, 0);
    all_w0 = visible_rows(r.n - 1, p.n_sink, p.window).w0;
    all_s1 = visible_rows(max(r.first, 0), p.n_sink, p.window).s1;
  }
  int st = 0;
  for (int u = tl.u0 + w; u < tl.u1; u += NW) {
    {
      const int nx = u + (G::NST - 1) * NW, ns = st == 0 ? G::NST - 1 : st - 1;
      if (nx < tl.u1) fetch(nx, ns, ahead);
      cp_async_commit();
      ahead = look_up(nx + NW);
    }
    cp_async_wait<G::NST - 1>();
    __syncwarp();
    const int r0 = tl.row(u);
    const uint32_t tk = ring + st * 2 * G::TILE;
    if (r0 + G::TK <= all_end && (r0 >= all_w0 || r0 + G::TK <= all_s1))
      tile(std::true_type{}, r0, tk);
    else
      tile(std::false_type{}, r0, tk);
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
  const bool bad = __syncthreads_or(!blocks_ok);
  const float down = __uint_as_float((127 - 20 + (lim >> 10)) << 23);  // 2^-k
  float* so = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float a0 = __shfl_sync(FULL_MASK, om[0], 4 * j + lt), a1 = __shfl_sync(FULL_MASK, om[1], 4 * j + lt);
    // the quarter's elements of this lane: d 128, two MMAs of two; d 64, one
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      const int e = j * (D / 4) + (lg & 3) * (D / 16) + (lg >> 2) * (D / 32) + 2 * i;
      const float(&y)[4] = o[j * (D / 64) + i];
#pragma unroll
      for (int c = 0; c < 4; ++c)
        so[(w * 8 + 2 * lt + (c & 1)) * RunSums<D>::HS + e + (c >> 1)] = fmaf(y[c], (c < 2 ? 0x1p24f : 0x1p20f) * down, (c & 1) ? a1 : a0);
    }
  }
  finish_run<Q4Tag, D, CHUNK>(p, r, tl, ls, split, pi, bad, so, sm_m, sm_l, run_ml);
}

}  // namespace
}  // namespace tri
