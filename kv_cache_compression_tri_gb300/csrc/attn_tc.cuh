// attn_tc.cuh -- what the tensor-core attention kernels share: tensor maps of
// the cache's rows, their copies into 128-byte-swizzled shared memory, and the
// bf16 forms of the tcgen05 operations in umma.cuh.
//
// A tile is 128 cached rows (or packed query rows) of D elements, held as D / 64
// columns of 64 elements: 128 bytes per row, 16 KB per column, the 16-byte
// chunks of row r permuted by chunk ^= (r % 8) -- what the tensor map's 128-byte
// swizzle writes. The same bytes serve as
//   - a K-major operand (rows = M or N, elements = K): 1024 bytes between groups
//     of eight rows, 32 bytes per MMA step of 16 elements;
//   - an MN-major operand (elements = N, rows = K): 64 elements of N per column,
//     16 KB between columns, 1024 bytes between groups of eight rows of K.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "attn_common.cuh"
#include "umma.cuh"

namespace tri {
namespace {

constexpr int TROWS = 128;          // rows of a tile
constexpr int TCOL = TROWS * 128;   // bytes of a 64-element column of it

constexpr int SMS = 152;

typedef CUresult (*Encode)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                           const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                           CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
// The driver's encoder, or NULL.
inline Encode tensor_map_encode() {
  static const Encode encode = [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      fn = nullptr;
    return reinterpret_cast<Encode>(fn);
  }();
  return encode;
}

// Where a layer's rows are, for the copy warps. Blocks (of a pool) or sequences, and heads, lie
// in any order and at any strides of whole 16 bytes. A tensor map of them as dimensions would
// ask each stride to be a multiple of the one before (so it is documented), so the maps are
// (element, row): a row's number is its offset divided by its size. Where strides are not
// whole rows (ODD) there is a map for each remainder, from the remainder on.
constexpr int MAX_ROW_MAPS = 16;  // 256-byte rows at offsets of whole 16 bytes
template <bool ODD>
struct RowMaps {
  CUtensorMap m[ODD ? MAX_ROW_MAPS : 1];
};
struct RowNumbers {
  int box_rows;          // rows of a box: 128, or a smaller block
  int odd;               // whether strides are not whole rows
  int64_t head, outer;   // from head to head, from block (or sequence) to the next: rows (int), if odd 16-byte units
  int none, row_mask;    // the number of no block (or sequence); row & row_mask is its place in the block
  int count;             // rows of the (first) map; one past its last row reads as zeros
};
// false: more rows than a coordinate can number.
inline bool row_numbers(const AttnParams& p, RowNumbers& r) {
  const RowMap& m = p.rows;
  const bool paged = m.table != nullptr;
  const int64_t n_outer = paged ? m.num_blocks : p.n_seq;
  const int64_t head = p.n_kv_heads > 1 ? (paged ? m.head_bytes : m.slice_bytes) : 0;
  const int64_t outer = n_outer > 1 ? (paged ? m.block_bytes : m.lh_count * m.slice_bytes) : 0;
  const int64_t count = ((p.n_kv_heads - 1) * head + (n_outer - 1) * outer) / m.row_bytes + (paged ? m.block_size : p.n_cap);
  r.odd = head % m.row_bytes != 0 || outer % m.row_bytes != 0;
  const int64_t unit = r.odd ? 16 : m.row_bytes;
  if (count > 0x7fffffff - 2 * TROWS) return false;
  r.none = paged ? m.num_blocks : -1;
  r.row_mask = paged ? m.block_size - 1 : 0x7fffffff;
  r.box_rows = paged && m.block_size < TROWS ? m.block_size : TROWS;
  r.head = head / unit;
  r.outer = outer / unit;
  r.count = static_cast<int>(count);
  return true;
}
// The tensor maps of `bytes` of rows from `base` on, boxes of 64 elements by box_rows rows.
template <bool ODD>
inline bool encode_row_maps(RowMaps<ODD>& maps, const void* base, int64_t bytes, int head_dim, int box_rows, Encode encode) {
  const int row_bytes = head_dim * 2;
  for (int i = 0; i < (ODD ? row_bytes / 16 : 1); ++i) {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(head_dim), static_cast<cuuint64_t>(std::max<int64_t>((bytes - 16 * i) / row_bytes, 1))};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(row_bytes)};
    const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t step[2] = {1, 1};
    if (encode(&maps.m[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, static_cast<char*>(const_cast<void*>(base)) + 16 * i, dims, strides, box,
               step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return false;
  }
  return true;
}
// Those of one layer's K (or V).
template <bool ODD>
inline bool encode_rows(RowMaps<ODD>& maps, const void* pool, const AttnParams& p, int head_dim, const RowNumbers& r, Encode encode) {
  const RowMap& m = p.rows;
  const int64_t base = p.layer * (m.table ? m.layer_bytes : p.n_kv_heads * m.slice_bytes);
  const int64_t n_outer = m.table ? m.num_blocks : p.n_seq, unit = ODD ? 16 : m.row_bytes;
  const int64_t bytes = ((p.n_kv_heads - 1) * r.head + (n_outer - 1) * r.outer) * unit +
                        static_cast<int64_t>(m.table ? m.block_size : p.n_cap) * m.row_bytes;
  return encode_row_maps(maps, static_cast<const char*>(pool) + base, bytes, head_dim, r.box_rows, encode);
}

__device__ __forceinline__ void tma_load2(uint32_t dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void tma_load4(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
          dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
      : "memory");
}

// The block that holds a lane's box of the tile at row k0 of sequence `seq` (num_blocks, which
// reads as zeros, where there is none), or for contiguous slices the sequence.
template <int D>
__device__ __forceinline__ int tile_block(const AttnParams& p, int box_rows, const int32_t* trow, int seq, int k0, int n, int lane) {
  if (!trow) return seq;
  const int i = lane / (D / 64), row = k0 + i * box_rows;
  if (i >= TROWS / box_rows || row >= n) return p.rows.num_blocks;
  const int blk = __ldg(trow + (row >> p.rows.block_shift));
  return blk < 0 || blk > p.rows.num_blocks ? p.rows.num_blocks : blk;
}
// A lane's box of a tile: 64 elements from `x` on of the rows from `row` on, at `off` in the tile.
template <int D>
struct LaneBox {
  int x, row;
  uint32_t off;
  bool live;
  __device__ __forceinline__ LaneBox(const RowNumbers& rn, int lane) {
    constexpr int COLS = D / 64;
    x = lane % COLS * 64;
    row = lane / COLS * rn.box_rows;
    off = lane % COLS * TCOL + row * 128;
    live = row < TROWS;
  }
};
// Where a lane's box of the tile at row k0 of head h is (blk as tile_block gave it): a row's
// number, and of which map. Worked out before the wait for a ring stage: after it, the dozen
// instructions are on the chain from a stage set free to its next rows (32 queries over 16
// caches of up to 32768 rows: 170 us, before it 164).
struct Place {
  int row, map;
};
template <int D, bool ODD>
__device__ __forceinline__ Place box_place(const RowNumbers& rn, const LaneBox<D>& box, int blk, int h, int k0) {
  const int row = (k0 + box.row) & rn.row_mask;
  if constexpr (ODD) {
    constexpr int UNITS = D / 8;  // 16-byte units of a row
    const int64_t at = blk * rn.outer + h * rn.head;
    return blk == rn.none ? Place{rn.count, 0} : Place{static_cast<int>(at / UNITS) + row, static_cast<int>(at % UNITS)};
  } else {
    return {blk == rn.none ? rn.count : blk * static_cast<int>(rn.outer) + h * static_cast<int>(rn.head) + row, 0};
  }
}
// A tile's cached rows of K or V into the tile at `dst`, by one warp, arriving once on `bar`.
// Rows past the slice are zeros or another slice's rows.
template <int D, bool ODD>
__device__ __forceinline__ void load_tile(uint32_t dst, const RowMaps<ODD>& maps, const LaneBox<D>& box, Place at, uint64_t* bar, int lane) {
  if (lane == 0) mbar_arrive_expect_tx(bar, D * 256);
  __syncwarp();
  if (box.live) tma_load2(dst + box.off, &maps.m[ODD ? at.map : 0], box.x, at.row, bar);
}

// Packed query rows of one tile (row u: token tok0 + u / group, head u % group;
// zeros from `rows` on), swizzled, by threads t of NT, as 16-byte asynchronous
// copies that have landed on return. (Through registers, with a division per
// row, a tile took 4 us of its CTA's time.)
template <int D, int NT>
__device__ __forceinline__ void load_query_tile(uint32_t dst, const AttnParams& p, int seq, int h, int tok0, int rows, int t) {
  constexpr int CH = D / 8, STEP = NT / CH;
  const int G = p.group, c = t % CH, dt = STEP / G, dg = STEP - dt * G;
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + seq * p.q_seq + tok0 * p.q_token + static_cast<int64_t>(h) * G * D;
  int u = t / CH, tok = u / G, g = u - tok * G;
#pragma unroll
  for (int i = 0; i < TROWS / STEP; ++i) {
    const bool live = u < rows;
    cp_async16(dst + (c >> 3) * TCOL + u * 128 + (((c & 7) ^ (u & 7)) << 4), live ? q + tok * p.q_token + g * D + c * 8 : q, live);
    u += STEP;
    tok += dt;
    g += dg;
    if (g >= G) {
      g -= G;
      ++tok;
    }
  }
  cp_async_commit();
  cp_async_wait<0>();
}

// kind::f16 with bf16 operands (bits 7-9 and 10-12 = 1), fp32 accumulation; bit
// 16: B is MN-major.
constexpr uint32_t bf16_idesc(int m, int n, bool b_mn) {
  return f16_idesc(m, n) | (1u << 7) | (1u << 10) | (b_mn ? 1u << 16 : 0u);
}
// Descriptor of an MN-major operand in the 128-byte swizzle: 16 KB between its
// 64-element columns (leading offset), 1024 bytes between groups of eight rows.
__device__ __forceinline__ uint64_t sw128_desc_mn(uint32_t saddr) {
  uint64_t d = static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(TCOL >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}
// D[tmem] (+)= A[tmem] * B[smem], A packed two bf16 per column.
__device__ __forceinline__ void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1 : 0)
      : "memory");
}
// 32 columns of this thread's lane.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
        "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Two fp32 operations in one instruction.
__device__ __forceinline__ void fma2(float& x0, float& x1, float a0, float a1, float b, float c) {
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %4};\n\tmov.b64 c, {%5, %5};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(x0), "=f"(x1) : "f"(a0), "f"(a1), "f"(b), "f"(c));
}
__device__ __forceinline__ void fma2(float& x0, float& x1, float a0, float a1, float b, float c0, float c1) {
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %4};\n\tmov.b64 c, {%5, %6};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(x0), "=f"(x1) : "f"(a0), "f"(a1), "f"(b), "f"(c0), "f"(c1));
}
__device__ __forceinline__ void add2(float& x0, float& x1, float a0, float a1) {
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%0, %1};\n\tadd.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "+f"(x0), "+f"(x1) : "f"(a0), "f"(a1));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Bit k of word i: column 32 i + k of a tile whose row 0 is cached row k0 is
// seen by the query at row r.
__device__ __forceinline__ uint32_t seen_bits(const AttnParams& p, int r, int k0, int i) {
  // columns [lo, hi) and [0, sink) of the word
  auto below = [](int n) { return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u; };
  const int c0 = k0 + 32 * i;
  const uint32_t upto = below(r + 1 - c0);
  if (p.window == 0) return upto;
  return upto & (~below(r + 1 - p.window - c0) | below(p.n_sink - c0));
}

// The 128-row tiles of the cache that rows r_lo (it may be negative) .. r_hi see: [0, a) and [b, e).
struct TileList {
  int a, b, e;
  __device__ __forceinline__ int count() const { return a + e - b; }
  __device__ __forceinline__ int at(int i) const { return i < a ? i : i - a + b; }
};
__device__ __forceinline__ TileList tiles_seen(const AttnParams& p, int r_lo, int r_hi) {
  if (r_hi < 0) return {0, 0, 0};
  TileList t;
  t.e = r_hi / TROWS + 1;
  if (p.window == 0) return {0, 0, t.e};
  t.a = (min(p.n_sink, r_hi + 1) + TROWS - 1) / TROWS;
  t.b = max(t.a, max(0, max(r_lo, 0) - p.window + 1) / TROWS);
  if (t.b > t.e) t.b = t.e;
  return t;
}

}  // namespace
}  // namespace tri
