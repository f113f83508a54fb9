// attn_prefill.cu -- causal attention of a chunk of new tokens over the cache,
// optionally windowed with first rows that stay visible.
#include <cuda_runtime.h>

#include "attn_tile.cuh"

namespace tri {
namespace {

template <int D>
struct PrefillSmem {
  float q[FM][D + 4];
  float k[FN][D + 4];
  float v[FN][D + 4];
  float w[FM][FN + 4];
  int flag;
};

template <typename T, int D>
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
  load_queries<T, D>(p, c, tok0, rows, sm.q);
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
    load_rows<T, D>(p, p.k, base, trow, k0, r_last, sm.k);
    load_rows<T, D>(p, p.v, base, trow, k0, r_last, sm.v);
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
    for (int e = 0; e < D / 16; ++e) static_cast<T*>(p.out)[head * D + tx + 16 * e] = from_f32<T>(o[a][e] * inv);
    if (p.lse && tx == 0) p.lse[head] = l[a] != 0.f ? LN2 * (m[a] + log2f(l[a])) : NEG_INF;
  }
}

template <typename T, int D>
cudaError_t launch_typed(const AttnParams& p, cudaStream_t st) {
  auto kern = prefill_kernel<T, D>;
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
  if (dt == TRI_BF16) return head_dim == 64 ? launch_typed<__nv_bfloat16, 64>(p, st) : launch_typed<__nv_bfloat16, 128>(p, st);
  return head_dim == 64 ? launch_typed<float, 64>(p, st) : launch_typed<float, 128>(p, st);
}

}  // namespace tri
