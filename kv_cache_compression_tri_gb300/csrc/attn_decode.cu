// attn_decode.cu -- attention of one new token per sequence over the cache,
// split over its length and joined, with the rows' accumulated weights.
//
// Per slice and query head g: x_j = scale * (q_g . k_j) over the visible rows,
// out_g = sum_j 2^(x_j - m) v_j / sum_j 2^(x_j - m). A slice's visible rows are
// cut into n_split equal runs, one CTA each; a CTA keeps a running maximum m,
// sum l and vector sum o per head (o and l rescaled when m grows), and writes
// (m, l, o) to the workspace. The join takes the largest m of a head's runs and
// adds the runs' l and o times 2^(m_run - m). Masses need every row's weight
// under the final log-sum, so the logits of the first pass are kept in the
// workspace and turned into weights by a third kernel.
#include <cuda_runtime.h>

#include "attn_common.cuh"

namespace tri {
namespace {

constexpr int DT = 128;   // threads per CTA
constexpr int LPR = 8;    // lanes per row
constexpr int GROUPS = DT / LPR;

// Row counts of the slice handled by this CTA; false: nothing to do. A slice
// with a fault is reported and its partial sums marked (sum -1).
struct Run {
  int64_t s;       // slice of the cache
  int n, seq, h;   // valid rows, sequence, KV head
  Visible vis;
  int count;       // visible rows
};

__device__ __forceinline__ bool slice_run(const AttnParams& p, int ls, Run& r) {
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
  r.vis = visible_rows(r.n - 1, p.n_sink, p.window);
  r.count = r.vis.s1 + r.n - r.vis.w0;
  return true;
}

template <typename T, int D, int GP>
__global__ void __launch_bounds__(DT) decode_partial_kernel(const __grid_constant__ AttnParams p) {
  constexpr int E = 16 / sizeof(T);       // elements per 16-byte chunk
  constexpr int C = D / (E * LPR);        // chunks per lane
  __shared__ float sq[GP][D];
  __shared__ float so[GROUPS][D];
  __shared__ float sm_m[GROUPS][GP], sm_l[GROUPS][GP];
  __shared__ int flag;
  const int split = blockIdx.x, ls = blockIdx.y, t = threadIdx.x, G = p.group;
  Run r;
  const int64_t pi = (static_cast<int64_t>(ls) * p.n_split + split) * G;
  bool ok = slice_run(p, ls, r);
  int i0 = 0, i1 = 0;
  const int32_t* trow = p.rows.seq_table(r.s);
  if (ok) {
    i0 = static_cast<int>(static_cast<int64_t>(r.count) * split / p.n_split);
    i1 = static_cast<int>(static_cast<int64_t>(r.count) * (split + 1) / p.n_split);
    const int shift = r.vis.w0 - r.vis.s1;
    bool blocks = p.rows.blocks_ok(trow, i0, min(i1, r.vis.s1), &flag);
    blocks = p.rows.blocks_ok(trow, max(i0, r.vis.s1) + shift, i1 + shift, &flag) && blocks;
    if (!blocks) {
      if (t == 0) set_status(p.dev_status, TRI_DEV_BAD_BLOCK);
      ok = false;
    }
  }
  if (!ok) {
    if (t < G) p.part_ml[pi + t] = make_float2(NEG_INF, -1.f);
    return;
  }
  const T* q = static_cast<const T*>(p.q) + r.seq * p.q_seq + static_cast<int64_t>(r.h) * G * D;
  for (int i = t; i < GP * D; i += DT) {
    const int g = i / D;
    sq[g][i % D] = g < G ? to_f32(q[i]) * (p.scale * LOG2E) : 0.f;
  }
  __syncthreads();
  const int rg = t / LPR, lane8 = t % LPR;
  float m[GP], l[GP], o[GP][C * E];
#pragma unroll
  for (int g = 0; g < GP; ++g) {
    m[g] = NEG_INF;
    l[g] = 0.f;
#pragma unroll
    for (int e = 0; e < C * E; ++e) o[g][e] = 0.f;
  }
  const int64_t base = p.rows.slice_base(r.s);
  float* logits = p.logits ? p.logits + static_cast<int64_t>(ls) * G * p.n_cap : nullptr;
  for (int i = i0 + rg; i - rg < i1; i += GROUPS) {
    const bool live = i < i1;
    const int j = i < r.vis.s1 ? i : i - r.vis.s1 + r.vis.w0;
    const int64_t off = live ? p.rows.row(base, trow, j) : 0;
    float x[GP];
#pragma unroll
    for (int g = 0; g < GP; ++g) x[g] = 0.f;
    uint4 vw[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      uint4 kw = make_uint4(0, 0, 0, 0);
      vw[c] = kw;
      if (live) {
        kw = __ldg(reinterpret_cast<const uint4*>(static_cast<const char*>(p.k) + off) + lane8 + LPR * c);
        vw[c] = __ldg(reinterpret_cast<const uint4*>(static_cast<const char*>(p.v) + off) + lane8 + LPR * c);
      }
      float kx[E];
      widen(kw, kx);
#pragma unroll
      for (int g = 0; g < GP; ++g)
#pragma unroll
        for (int e = 0; e < E; ++e) x[g] = fmaf(sq[g][(lane8 + LPR * c) * E + e], kx[e], x[g]);
    }
#pragma unroll
    for (int g = 0; g < GP; ++g) {
#pragma unroll
      for (int w = LPR / 2; w >= 1; w >>= 1) x[g] += __shfl_xor_sync(FULL_MASK, x[g], w);
      if (!live) x[g] = NEG_INF;
      if (logits && live && lane8 == g % LPR && g < G) logits[static_cast<int64_t>(g) * p.n_cap + j] = x[g];
      const float mn = fmaxf(m[g], x[g]);
      const float mu = mn == NEG_INF ? 0.f : mn;
      const float a = fast_exp2(m[g] - mu), w = fast_exp2(x[g] - mu);
      m[g] = mn;
      l[g] = fmaf(l[g], a, w);
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float vx[E];
        widen(vw[c], vx);
#pragma unroll
        for (int e = 0; e < E; ++e) o[g][c * E + e] = fmaf(o[g][c * E + e], a, w * vx[e]);
      }
    }
  }
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
      p.part_o[(pi + g) * D + e] = sum;
    }
    if (t == 0) {
      float sum = 0.f;
      for (int u = 0; u < GROUPS; ++u) sum = fmaf(sm_l[u][g], fast_exp2(sm_m[u][g] - mu), sum);
      p.part_ml[pi + g] = make_float2(mx, sum);
    }
  }
}

// Joined (m, l) of a head's runs; false: skipped.
__device__ __forceinline__ bool join_ml(const AttnParams& p, int ls, int g, float& m, float& l) {
  const float2* ml = p.part_ml + static_cast<int64_t>(ls) * p.n_split * p.group + g;
  m = NEG_INF;
  l = 0.f;
  for (int i = 0; i < p.n_split; ++i) {
    const float2 x = ml[static_cast<int64_t>(i) * p.group];
    if (x.y < 0.f) return false;
    m = fmaxf(m, x.x);
  }
  const float mu = m == NEG_INF ? 0.f : m;
  for (int i = 0; i < p.n_split; ++i) {
    const float2 x = ml[static_cast<int64_t>(i) * p.group];
    l = fmaf(x.y, fast_exp2(x.x - mu), l);
  }
  return true;
}

template <typename T, int D>
__global__ void __launch_bounds__(D) decode_join_kernel(const __grid_constant__ AttnParams p) {
  const int ls = blockIdx.x / p.group, g = blockIdx.x % p.group, t = threadIdx.x;
  const int seq = ls / p.n_kv_heads, h = ls % p.n_kv_heads;
  float m, l;
  if (!join_ml(p, ls, g, m, l)) return;
  const float mu = m == NEG_INF ? 0.f : m;
  float o = 0.f;
  for (int i = 0; i < p.n_split; ++i) {
    const int64_t pi = (static_cast<int64_t>(ls) * p.n_split + i) * p.group + g;
    o = fmaf(p.part_o[pi * D + t], fast_exp2(p.part_ml[pi].x - mu), o);
  }
  const int64_t row = (static_cast<int64_t>(seq) * p.n_kv_heads + h) * p.group + g;
  static_cast<T*>(p.out)[row * D + t] = from_f32<T>(l != 0.f ? o / l : 0.f);
  if (p.lse && t == 0) p.lse[row] = l != 0.f ? LN2 * (m + log2f(l)) : NEG_INF;
}

// mass[j] += sum over the heads of 2^(x_j - m) / l.
__global__ void __launch_bounds__(256) decode_mass_kernel(const __grid_constant__ AttnParams p) {
  __shared__ float lse2[MAX_GROUP];
  __shared__ int skip;
  const int ls = blockIdx.y, t = threadIdx.x;
  Run r;
  if (!slice_run(p, ls, r)) return;
  if (t == 0) skip = 0;
  __syncthreads();
  if (t < p.group) {
    float m, l;
    if (!join_ml(p, ls, t, m, l)) skip = 1;
    lse2[t] = m + log2f(l);
  }
  __syncthreads();
  if (skip) return;
  const float* logits = p.logits + static_cast<int64_t>(ls) * p.group * p.n_cap;
  float* mass = p.mass + r.s * p.n_cap;
  for (int i = blockIdx.x * 256 + t; i < r.count; i += gridDim.x * 256) {
    const int j = i < r.vis.s1 ? i : i - r.vis.s1 + r.vis.w0;
    float w = 0.f;
    for (int g = 0; g < p.group; ++g) w += fast_exp2(logits[static_cast<int64_t>(g) * p.n_cap + j] - lse2[g]);
    mass[j] += w;
  }
}

template <typename T, int D>
cudaError_t launch_typed(const AttnParams& p, cudaStream_t st) {
  const int n = p.n_seq * p.n_kv_heads;
  const dim3 grid(static_cast<unsigned>(p.n_split), static_cast<unsigned>(n));
  if (p.group == 1) decode_partial_kernel<T, D, 1><<<grid, DT, 0, st>>>(p);
  else if (p.group == 2) decode_partial_kernel<T, D, 2><<<grid, DT, 0, st>>>(p);
  else if (p.group <= 4) decode_partial_kernel<T, D, 4><<<grid, DT, 0, st>>>(p);
  else decode_partial_kernel<T, D, 8><<<grid, DT, 0, st>>>(p);
  note_launch();
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  decode_join_kernel<T, D><<<static_cast<unsigned>(n * p.group), D, 0, st>>>(p);
  note_launch();
  e = cudaGetLastError();
  if (e != cudaSuccess || !p.mass) return e;
  decode_mass_kernel<<<grid, 256, 0, st>>>(p);
  note_launch();
  return cudaGetLastError();
}

}  // namespace

int attn_decode_splits(int n_slices, int max_rows) {
  const int want = (152 * 8 + n_slices - 1) / n_slices;
  const int most = (max_rows + 127) / 128;
  return want < 1 ? 1 : (want < most ? want : most);
}

cudaError_t launch_attn_decode(const AttnParams& p, tri_dtype dt, int head_dim, cudaStream_t st) {
  if (dt == TRI_BF16) return head_dim == 64 ? launch_typed<__nv_bfloat16, 64>(p, st) : launch_typed<__nv_bfloat16, 128>(p, st);
  return head_dim == 64 ? launch_typed<float, 64>(p, st) : launch_typed<float, 128>(p, st);
}

}  // namespace tri
