// q4_rows.cu -- one layer's rows of a 4-bit cache written out: for the caller
// (tri_read_rows, bf16), or for a chunk's attention, which then runs on them
// (tri_attn_prefill_q4: K as a bf16 pair, V in fp16. With both rounded to bf16 once, log-sums
// were off by 1e-5 to 7e-5 of themselves, and results by more than twice what their own
// rounding leaves).
//
// A thread writes 16 bytes of each: eight elements of one quarter, minimum + scale * code.
// Bound: HBM, d / 2 + 16 bytes in and 2 d (4 d of a pair) out per row (a prompt's rows stay in
// L2 for the attention that follows).
//
// For a chunk: rows out of every query's sight are zero where a 128-row tile holds rows in
// sight (the attention's weights there are 0, which a NaN would survive) and not
// written elsewhere; and the first CTA of a sequence checks every table entry that
// its queries need, so that the attention leaves the sequence out when one is bad.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "attn_common.cuh"
#include "q4_common.cuh"

namespace tri {
namespace {

constexpr int RT = 256;    // threads per CTA
constexpr int CHUNK = 64;  // rows of a CTA, K and V
constexpr int SIGHT = 128; // rows that an attention tile reads together

// Elements 8 c .. 8 c + 7 of a 4-bit row: their words, and their quarter's pair.
struct Eight {
  uint32_t a, b, pair;
};
template <int D>
__device__ __forceinline__ Eight load8(const char* row, int c) {
  const int j = c / (D / 32);  // quarter
  const uint32_t* words = reinterpret_cast<const uint32_t*>(row);
  Eight x;
  x.pair = __ldg(reinterpret_cast<const uint32_t*>(row + Q4Row<D>::CODES) + j);
  if constexpr (D == 128) {
    x.a = __ldg(words + 4 * (c & 3) + j);
    x.b = 0;
  } else {
    // of lanes 2 (c & 1) and the next
    x.a = __ldg(words + 4 * (c & 1) + (j >> 1));
    x.b = __ldg(words + 4 * (c & 1) + 2 + (j >> 1));
  }
  return x;
}
template <int D>
__device__ __forceinline__ void values8(const Eight& w, int c, float (&x)[8]) {
  const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w.pair));  // scale, minimum
  uint32_t n = w.a;  // the eight codes, in order
  // (d 64: four codes of a word each, in its bytes j & 1 and 2 + (j & 1))
  if constexpr (D == 64) n = __byte_perm(w.a, w.b, (c >> 1) & 1 ? 0x7531 : 0x6420);
  // (a half with exponent 0 and c in its low bits is c 2^-24, four bits higher c 2^-20: exact)
  const float s0 = p.x * 0x1p24f, s1 = p.x * 0x1p20f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t pair = (e & 2 ? n >> 8 : n) & (e & 1 ? 0x00f000f0u : 0x000f000fu);  // codes e and e + 4
    const float2 c = __half22float2(*reinterpret_cast<const __half2*>(&pair));
    x[e] = fmaf(c.x, e & 1 ? s1 : s0, p.y);
    x[e + 4] = fmaf(c.y, e & 1 ? s1 : s0, p.y);
  }
}
__device__ __forceinline__ uint4 bf16_of(const float (&x)[8]) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}
// What rounding to `hi` left.
__device__ __forceinline__ uint4 rest_of(const float (&x)[8], uint4 hi) {
  const uint32_t h[4] = {hi.x, hi.y, hi.z, hi.w};
  uint32_t r[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) r[k] = pack_bf16(x[2 * k] - bf16_lo(h[k]), x[2 * k + 1] - bf16_hi(h[k]));
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// Rows of a slice of n that some of its nn newest queries see: [0, s1) and [w0, n).
__device__ __forceinline__ Visible chunk_sight(const Q4RowsParams& p, int n, int nn) {
  return {visible_rows(n - 1, p.n_sink, p.window).s1, visible_rows(max(n - nn, 0), p.n_sink, p.window).w0};
}

template <int D, bool CHUNKED>
__global__ void __launch_bounds__(RT) q4_rows_kernel(const __grid_constant__ Q4RowsParams p, int tiles) {
  constexpr int LPR = D / 8;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tile = blockIdx.x % tiles, ls = blockIdx.x / tiles;
  const int seq = ls / p.n_kv_heads, h = ls % p.n_kv_heads;
  const int64_t s0 = (static_cast<int64_t>(seq) * p.n_layers + p.layer) * p.n_kv_heads, s = s0 + h;
  const int n = p.n_valid[s], nn = !CHUNKED ? 0 : p.n_new ? __ldg(p.n_new + seq) : p.n_q;
  const int32_t* trow = p.rows.seq_table(s);
  if (CHUNKED && tile == 0) {
    if (threadIdx.x == 0) p.n_valid_out[ls] = n;
    if (h == 0) {
      bool bad = nn < 0 || nn > p.n_q;
      if (bad && threadIdx.x == 0) set_status(p.dev_status, TRI_DEV_BAD_QUERY);
      if (trow && !bad && nn > 0) {
        int last = -1;
        for (int k = 0; k < p.n_kv_heads; ++k) {
          const int nk = p.n_valid[s0 + k];
          if (nk == last || nk <= 0 || nk > p.n_cap) continue;  // (a bad count is the attention's to report)
          last = nk;
          const Visible vis = chunk_sight(p, nk, nn);
          const int b1 = (nk - 1) >> p.rows.block_shift, bw = vis.w0 >> p.rows.block_shift;
          const int bs = vis.s1 > 0 ? (vis.s1 - 1) >> p.rows.block_shift : -1;
          for (int b = threadIdx.x; b <= b1; b += RT) {
            if (b > bs && b < bw) continue;
            const int blk = __ldg(trow + b);
            bad |= blk < 0 || blk >= p.rows.num_blocks;
          }
        }
        bad = __syncthreads_or(bad);
        if (bad && threadIdx.x == 0) set_status(p.dev_status, TRI_DEV_BAD_BLOCK);
      }
      if (threadIdx.x == 0) p.n_new_out[seq] = bad ? 0 : nn;
    }
  }
  if (n < 0 || n > p.n_cap) {
    if (!CHUNKED && threadIdx.x == 0) set_status(p.dev_status, TRI_DEV_NVALID_OVER_CAP);
    return;
  }
  const int r0 = tile * CHUNK, r1 = n - r0 > CHUNK ? r0 + CHUNK : n;
  if (r0 >= r1 || (CHUNKED && nn <= 0)) return;
  Visible vis{0, 0};
  if constexpr (CHUNKED) {
    vis = chunk_sight(p, n, nn);
    if (r0 >= (vis.s1 + SIGHT - 1) / SIGHT * SIGHT && r1 <= vis.w0 / SIGHT * SIGHT) return;
  }
  const int64_t base = p.rows.slice_base(s);
  const int c = threadIdx.x % LPR;
  const int64_t out = static_cast<int64_t>(ls) * p.n_cap;
  // all loads of the thread, then its stores
  constexpr int N = CHUNK * LPR / RT;
  Eight w[N][2];
  uint32_t write = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int r = r0 + i * (RT / LPR) + static_cast<int>(threadIdx.x) / LPR;
    bool ok = r < r1 && (!CHUNKED || r < vis.s1 || r >= vis.w0);
    int64_t off = base + static_cast<int64_t>(r) * p.rows.row_bytes;
    if (trow && ok) {
      const int blk = __ldg(trow + (r >> p.rows.block_shift));
      ok = blk >= 0 && blk < p.rows.num_blocks;
      if (!CHUNKED && !ok) set_status(p.dev_status, TRI_DEV_BAD_BLOCK);
      off = base + blk * p.rows.block_bytes + static_cast<int64_t>(r & (p.rows.block_size - 1)) * p.rows.row_bytes;
    }
    if (r < r1 && (CHUNKED || ok)) write |= 1u << i;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      w[i][kv] = {0, 0, 0};  // (reads as zeros)
      if (ok && p.dst[kv]) w[i][kv] = load8<D>(p.src[kv] + off, c);
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int r = r0 + i * (RT / LPR) + static_cast<int>(threadIdx.x) / LPR;
    if (!(write >> i & 1)) continue;
    const int64_t to = (out + r) * (D / 8) + c;
    float x[8];
    if (p.dst[0]) {
      values8<D>(w[i][0], c, x);
      const uint4 hi = bf16_of(x);
      static_cast<uint4*>(p.dst[0])[to] = hi;
      if (CHUNKED) static_cast<uint4*>(p.k_rest)[to] = rest_of(x, hi);
    }
    if (p.dst[1]) {
      values8<D>(w[i][1], c, x);
      static_cast<uint4*>(p.dst[1])[to] =
          CHUNKED ? make_uint4(pack_half(x[0], x[1]), pack_half(x[2], x[3]), pack_half(x[4], x[5]), pack_half(x[6], x[7])) : bf16_of(x);
    }
  }
}

}  // namespace

cudaError_t launch_q4_rows(const Q4RowsParams& p, int head_dim, cudaStream_t st) {
  const int tiles = (p.n_cap - 1) / CHUNK + 1;
  const int64_t ctas = static_cast<int64_t>(p.n_seq) * p.n_kv_heads * tiles;
  if (ctas > 0x7fffffff) return cudaErrorNotSupported;  // (more than a launch counts)
  auto kern = head_dim == 64 ? (p.n_new_out ? q4_rows_kernel<64, true> : q4_rows_kernel<64, false>)
                             : (p.n_new_out ? q4_rows_kernel<128, true> : q4_rows_kernel<128, false>);
  kern<<<static_cast<unsigned>(ctas), RT, 0, st>>>(p, tiles);
  note_launch();
  return cudaGetLastError();
}

}  // namespace tri
