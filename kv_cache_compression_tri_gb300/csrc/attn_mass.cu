// attn_mass.cu -- the accumulated weight of every cached row under a chunk of
// queries: mass[j] += sum over the queries that see row j of e^(x_j - lse).
// A CTA owns a run of cached rows and goes over the chunk's queries, so each
// mass is summed by one thread row in a fixed order and written once.
#include <cuda_runtime.h>

#include "attn_tile.cuh"

namespace tri {
namespace {

template <int D>
struct MassSmem {
  float q[FM][D + 4];
  float k[FN][D + 4];
  float lse2[FM];
  float part[16][FN];
  int flag;
};

template <typename T, int D>
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
  if (!p.rows.blocks_ok(trow, k0, last + 1, &sm.flag)) {
    if (t == 0) set_status(p.dev_status, TRI_DEV_BAD_BLOCK);
    return;
  }
  load_rows<T, D>(p, p.k, base, trow, k0, last, sm.k);
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
  const int tpt = FM / G;
  for (int tok0 = 0; tok0 < c.n_new; tok0 += tpt) {
    const int toks = min(tpt, c.n_new - tok0), rows = toks * G, r_first = c.r0 + tok0;
    if (!tile_seen(p, k0, FN, max(r_first, 0), r_first + toks - 1)) continue;
    __syncthreads();
    load_queries<T, D>(p, c, tok0, rows, sm.q);
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

template <typename T, int D>
cudaError_t launch_typed(const AttnParams& p, cudaStream_t st) {
  auto kern = mass_kernel<T, D>;
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
  if (dt == TRI_BF16) return head_dim == 64 ? launch_typed<__nv_bfloat16, 64>(p, st) : launch_typed<__nv_bfloat16, 128>(p, st);
  return head_dim == 64 ? launch_typed<float, 64>(p, st) : launch_typed<float, 128>(p, st);
}

}  // namespace tri
