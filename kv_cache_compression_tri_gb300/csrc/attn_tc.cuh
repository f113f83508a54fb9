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

// Tensor map of one layer's K (or V) rows: (element, row, head, sequence) of
// contiguous slices, (element, row of the block, head, block) of a pool. Boxes
// of 64 elements by up to 128 rows. Returns the rows of a box, 0 on failure.
inline int encode_rows(CUtensorMap* map, const void* pool, const AttnParams& p, int head_dim, Encode encode) {
  const RowMap& m = p.rows;
  const bool paged = m.table != nullptr;
  const int64_t base = p.layer * (paged ? m.layer_bytes : p.n_kv_heads * m.slice_bytes);
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(head_dim), static_cast<cuuint64_t>(paged ? m.block_size : p.n_cap),
                              static_cast<cuuint64_t>(p.n_kv_heads), static_cast<cuuint64_t>(paged ? m.num_blocks : p.n_seq)};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(m.row_bytes), static_cast<cuuint64_t>(paged ? m.head_bytes : m.slice_bytes),
                           static_cast<cuuint64_t>(paged ? m.block_bytes : m.lh_count * m.slice_bytes)};
  if (dims[3] == 1 && strides[2] < strides[1]) strides[2] = strides[1];  // (never used)
  const int rows = paged && m.block_size < TROWS ? m.block_size : TROWS;
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(rows), 1, 1};
  const cuuint32_t step[4] = {1, 1, 1, 1};
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, static_cast<char*>(const_cast<void*>(pool)) + base, dims,
                            strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? rows : 0;
}

__device__ __forceinline__ void tma_load4(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
          dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
      : "memory");
}

// Block that holds a lane's box of the tile at row k0 (pools only): num_blocks,
// which the map fills with zeros, where there is none.
template <int D>
__device__ __forceinline__ int tile_block(const AttnParams& p, int box_rows, const int32_t* trow, int k0, int n, int lane) {
  const int i = lane / (D / 64), row = k0 + i * box_rows;
  if (!trow || i >= TROWS / box_rows || row >= n) return p.rows.num_blocks;
  const int blk = __ldg(trow + (row >> p.rows.block_shift));
  return blk < 0 || blk > p.rows.num_blocks ? p.rows.num_blocks : blk;
}
// Cached rows [k0, k0 + 128) of slice (seq, h) into the tile at `dst`, by the
// lanes of one warp after one of them expected D * 256 bytes on `bar`; blk as
// tile_block gave it. Rows past the cache read as zeros too.
template <int D>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* map, const AttnParams& p, int box_rows, bool paged, int blk,
                                          int seq, int h, int k0, uint64_t* bar, int lane) {
  constexpr int COLS = D / 64;
  if (lane >= TROWS / box_rows * COLS) return;
  const int col = lane % COLS, i = lane / COLS, row = k0 + i * box_rows;
  const uint32_t d = dst + col * TCOL + i * box_rows * 128;
  if (paged) tma_load4(d, map, 64 * col, row & (p.rows.block_size - 1), h, blk, bar);
  else tma_load4(d, map, 64 * col, row, h, seq, bar);
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
