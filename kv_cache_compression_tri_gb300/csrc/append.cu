// append.cu -- new tokens into one layer of the cache, rotated on the way.
//
// Token i of a sequence becomes row n_valid + i of the layer's slices: V as it is,
// K (and the queries, into a buffer of their own) with band f multiplied by
// e^{i w_f p}. p is one of the token's positions, the one of the band's axis. The
// phase p w_f / 2 pi is a 64-bit fixed-point product, exact modulo a turn, so
// far positions keep their angle.
//
// Bound: every row is read once and written once, so HBM. A warp takes one token
// and a run of KV heads with their query heads, since the token's sines serve all
// of them: 2 or 4 bands a lane (40 instructions each), then about 50
// instructions per 256-byte row. A lane has four elements of a row: 8 or 16
// bytes, a whole row of d 128 per load instruction, two rows of d 64. With
// rotation in halves an element's partner sits 16 (8) lanes on and comes by a
// shuffle.
//
// 4-bit rows: a quarter's minimum and maximum are shuffles over 8 (4) lanes.
// Which fp16 or code is nearest is decided as in 64 bits: a lane bounds the error
// of its fp32 arithmetic, and where a border lies within it, the warp repeats the
// row in fp64 (a few rows in a thousand; all rows in fp64 would be bound by the
// fp64 units, 1/60 of the fp32 rate).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "attn_common.cuh"
#include "q4_common.cuh"

namespace tri {
namespace {

constexpr int AW = 8;      // warps per CTA
constexpr int BATCH = 4;   // rows whose loads a lane has in flight

// The rotation of a lane's bands at the token's positions.
template <int NB>
struct Turns {
  float c[NB], s[NB];
};

// cos and sin of 2 pi frac(x nu): sincospi of the phase rounded to fp32, and the first-order
// step for what the rounding left (error about 2^-23).
__device__ __forceinline__ void turn(int32_t x, uint64_t nu, float& c, float& s) {
  const int32_t hi = static_cast<int32_t>((static_cast<uint64_t>(static_cast<int64_t>(x)) * nu) >> 32);  // 2^-32 turns
  const float h = static_cast<float>(hi);
  const float rest = static_cast<float>(hi - static_cast<int32_t>(h)) * 1.4629180792671596e-09f;  // radians: 2 pi 2^-32
  float s0, c0;
  sincospif(h * 4.656612873077393e-10f, &s0, &c0);  // half turns: 2^-31
  c = fmaf(-s0, rest, c0);
  s = fmaf(c0, rest, s0);
}

// Band of a lane's b-th rotation: interleaved, bands 2 l and 2 l + 1; in halves, the four of its elements.
template <int D, bool HALF>
__device__ __forceinline__ int band_of(int l, int b) {
  return HALF ? (4 * l) % (D / 2) + b : 2 * l + b;
}
__device__ __forceinline__ int32_t position_of(const AppendParams& p, const int32_t* at, int f) {
  const int a = (p.axis_bits[f >> 4] >> (2 * (f & 15))) & 3;
  return __ldg(at + a);
}

// x rotated in place; `other` the lane of the partner elements (halves).
template <int D, bool HALF, typename R, int NB>
__device__ __forceinline__ void rotate(R (&x)[4], const R (&c)[NB], const R (&s)[NB], int l) {
  if constexpr (HALF) {
    const R sign = l < D / 8 ? R(-1) : R(1);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const R y = __shfl_xor_sync(FULL_MASK, x[e], D / 8);
      x[e] = x[e] * c[e] + sign * y * s[e];
    }
  } else {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const R re = x[2 * b], im = x[2 * b + 1];
      x[2 * b] = re * c[b] - im * s[b];
      x[2 * b + 1] = re * s[b] + im * c[b];
    }
  }
}

// A lane's part of a row: four codes, and its quarter's pair.
struct Quad {
  uint32_t code[4];
  __half scale, low;
};

// The row's quarter in fp64 (x: before the rotation).
template <int D, bool HALF, bool ROT>
__device__ __noinline__ Quad quantise64(const AppendParams& p, const int32_t* at, float4 xin, int l) {
  double x[4] = {xin.x, xin.y, xin.z, xin.w};
  if constexpr (ROT) {
    constexpr int NB = HALF ? 4 : 2;
    double c[NB], s[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int f = band_of<D, HALF>(l, b);
      const int64_t t = static_cast<int64_t>(static_cast<uint64_t>(static_cast<int64_t>(position_of(p, at, f))) * p.nu[f]);
      sincospi(static_cast<double>(t) * 0x1p-63, &s[b], &c[b]);
    }
    rotate<D, HALF>(x, c, s, l);
  }
  double lo = Q4_MOST, hi = -Q4_MOST;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[e] = fmin(fmax(x[e], -static_cast<double>(Q4_MOST)), static_cast<double>(Q4_MOST));
    lo = fmin(lo, x[e]);
    hi = fmax(hi, x[e]);
  }
#pragma unroll
  for (int k = D / 32; k >= 1; k >>= 1) {
    lo = fmin(lo, __shfl_xor_sync(FULL_MASK, lo, k));
    hi = fmax(hi, __shfl_xor_sync(FULL_MASK, hi, k));
  }
  Quad q;
  q.low = __double2half(lo);
  const double m = static_cast<double>(__half2float(q.low));
  q.scale = __double2half(fmax(hi - m, 0.0) / 15.0);
  const double sc = static_cast<double>(__half2float(q.scale));
#pragma unroll
  for (int e = 0; e < 4; ++e) q.code[e] = sc > 0.0 ? static_cast<uint32_t>(fmin(fmax(rint((x[e] - m) / sc), 0.0), 15.0)) : 0u;
  return q;
}

// The row's quarter; x0: before the rotation, x: after it.
template <int D, bool HALF, bool ROT>
__device__ __forceinline__ Quad quantise(const AppendParams& p, const int32_t* at, const float (&x0)[4], float (&x)[4], int l) {
  float lo = Q4_MOST, hi = -Q4_MOST, err = 0.f;
  bool nan = false;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    nan |= x[e] != x[e];
    if constexpr (ROT) err = fmaxf(err, fabsf(x0[e]));
    x[e] = fminf(fmaxf(x[e], -Q4_MOST), Q4_MOST);
    lo = fminf(lo, x[e]);
    hi = fmaxf(hi, x[e]);
  }
  if constexpr (ROT && HALF) err = fmaxf(err, __shfl_xor_sync(FULL_MASK, err, D / 8));
#pragma unroll
  for (int k = D / 32; k >= 1; k >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(FULL_MASK, lo, k));
    hi = fmaxf(hi, __shfl_xor_sync(FULL_MASK, hi, k));
    if constexpr (ROT) err = fmaxf(err, __shfl_xor_sync(FULL_MASK, err, k));
  }
  constexpr int LANES = D / 16;  // of a quarter
  const unsigned quarter = ((1u << LANES) - 1) << ((threadIdx.x & 31) / LANES * LANES);
  nan = (__ballot_sync(FULL_MASK, nan) & quarter) != 0;
  // a rotated element errs by at most 2^-21 of the larger of its two inputs (the sines by 2^-22, three roundings)
  err = fminf(err, 2 * Q4_MOST) * 0x1p-21f;
  Quad q;
  q.low = __float2half_rn(lo);
  bool border = false;
  if constexpr (ROT) border = __half_as_ushort(__float2half_rn(lo - err)) != __half_as_ushort(__float2half_rn(lo + err));
  const float m = __half2float(q.low), span = fmaxf(hi - m, 0.f), es = err + span * 0x1p-22f;
  q.scale = __float2half_rn(span * (1.f / 15.f));
  border |= __half_as_ushort(__float2half_rn(fmaxf(span - es, 0.f) * (1.f / 15.f))) !=
            __half_as_ushort(__float2half_rn((span + es) * (1.f / 15.f)));
  const float sc = __half2float(q.scale), inv = sc > 0.f ? 1.f / sc : 0.f;
  // (codes err by the element's error over the scale, and 2^-18 for the arithmetic on up to 16)
  const float ec = fmaf(err, inv, 0x1p-18f);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float u = (x[e] - m) * inv, c = rintf(u);
    border |= fabsf(u - c) > 0.5f - ec;
    q.code[e] = static_cast<uint32_t>(fminf(fmaxf(c, 0.f), 15.f));
  }
  if (__any_sync(FULL_MASK, border && !nan)) q = quantise64<D, HALF, ROT>(p, at, make_float4(x0[0], x0[1], x0[2], x0[3]), l);
  if (nan) {
    q.low = q.scale = __ushort_as_half(0x7fff);
#pragma unroll
    for (int e = 0; e < 4; ++e) q.code[e] = 0;
  }
  return q;
}

// A lane's four elements 4 l .. 4 l + 3 to the 4-bit row at `row`.
template <int D>
__device__ __forceinline__ void store_quad(char* row, const Quad& q, int l) {
  const uint32_t c01 = q.code[0] | q.code[1] << 4, c23 = q.code[2] | q.code[3] << 4;
  if constexpr (D == 128) {
    const int j = l >> 3, t = (l & 7) >> 1;
    *reinterpret_cast<uint16_t*>(row + 4 * (4 * t + j) + 2 * (l & 1)) = static_cast<uint16_t>(c01 | c23 << 8);
  } else {
    const int j = l >> 2, t = l & 3;
    char* w = row + 4 * (2 * t + (j >> 1)) + (j & 1);
    w[0] = static_cast<char>(c01);
    w[2] = static_cast<char>(c23);
  }
  constexpr int LANES = D / 16;
  if (l % LANES == 0) *reinterpret_cast<__half2*>(row + Q4Row<D>::CODES + 4 * (l / LANES)) = __halves2half2(q.scale, q.low);
}

template <typename T>
struct Raw;  // four elements as loaded
template <>
struct Raw<__nv_bfloat16> {
  uint2 w;
  __device__ __forceinline__ void get(float (&x)[4]) const {
    x[0] = bf16_lo(w.x);
    x[1] = bf16_hi(w.x);
    x[2] = bf16_lo(w.y);
    x[3] = bf16_hi(w.y);
  }
  __device__ __forceinline__ void set(const float (&x)[4]) { w = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])); }
};
template <>
struct Raw<float> {
  float4 w;
  __device__ __forceinline__ void get(float (&x)[4]) const {
    x[0] = w.x;
    x[1] = w.y;
    x[2] = w.z;
    x[3] = w.w;
  }
  __device__ __forceinline__ void set(const float (&x)[4]) { w = make_float4(x[0], x[1], x[2], x[3]); }
};

__device__ __forceinline__ int append_tokens(const AppendParams& p, int seq) {
  const int n = p.n_new ? __ldg(p.n_new + seq) : p.n_q;
  if (n < 0 || n > p.n_q) {
    set_status(p.dev_status, TRI_DEV_BAD_QUERY);
    return -1;
  }
  return n;
}
__device__ __forceinline__ int64_t append_slice(const AppendParams& p, int seq, int h) {
  return (static_cast<int64_t>(seq) * p.n_layers + p.layer) * p.n_kv_heads + h;
}
// Whether nn rows fit behind the n of a slice.
__device__ __forceinline__ bool rows_fit(const AppendParams& p, int n, int nn) {
  if (n >= 0 && n <= p.n_cap && nn <= p.n_cap - n) return true;
  set_status(p.dev_status, TRI_DEV_NVALID_OVER_CAP);
  return false;
}

template <typename T, int D, bool HALF, bool Q4>
__global__ void __launch_bounds__(AW * 32) append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int LPR = D / 4, RPW = 32 / LPR, NB = HALF ? 4 : 2;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane / LPR, l = lane % LPR;
  int b = blockIdx.x;
  const int ht = b % p.head_tiles;
  b /= p.head_tiles;
  const int tt = b % p.token_tiles, seq = b / p.token_tiles;
  const int head_ways = AW / p.token_ways;
  const int i = tt * p.token_ways + w / head_ways;
  const int hpw = p.heads_per_warp;
  const int h0 = (ht * head_ways + w % head_ways) * hpw, hc = min(hpw, p.n_kv_heads - h0);  // (may be none)
  const int nn = append_tokens(p, seq);
  if (i < nn && hc > 0) {
    // where the heads' rows go: byte offset in K and V, -1 for none (lane j: head h0 + j)
    int64_t dst = -1;
    const int32_t* at = p.positions + (static_cast<int64_t>(seq) * p.n_q + i) * p.n_axes;
    if (lane < hc) {
      const int64_t s = append_slice(p, seq, h0 + lane);
      const int n = p.n_valid[s];
      if (rows_fit(p, n, nn)) {
        const int row = n + i;
        bool ok = true;
        if (p.rows.paged()) {
          const int blk = __ldg(p.rows.seq_table(s) + (row >> p.rows.block_shift));
          ok = blk >= 0 && blk < p.rows.num_blocks;
          if (!ok) set_status(p.dev_status, TRI_DEV_BAD_BLOCK);
        }
        if (ok) {
          dst = p.rows.row(p.rows.slice_base(s), p.rows.seq_table(s), row);
          if (p.pos) p.pos[s * p.n_cap + row] = __ldg(at);
        }
      }
    }
    Turns<NB> tn;
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      const int f = band_of<D, HALF>(l, k);
      turn(position_of(p, at, f), p.nu[f], tn.c[k], tn.s[k]);
    }
    // K and V rows: BATCH / 2 pairs of them in flight
    const T* kn = static_cast<const T*>(p.kn) + seq * p.k_seq + i * p.k_token + static_cast<int64_t>(h0) * D + 4 * l;
    const T* vn = static_cast<const T*>(p.vn) + seq * p.v_seq + i * p.v_token + static_cast<int64_t>(h0) * D + 4 * l;
    for (int r0 = 0; r0 < hc; r0 += BATCH / 2 * RPW) {
      Raw<T> xk[BATCH / 2], xv[BATCH / 2];
#pragma unroll
      for (int k = 0; k < BATCH / 2; ++k) {
        const int r = r0 + k * RPW + sub;
        if (r < hc) {
          xk[k].w = __ldg(reinterpret_cast<const decltype(xk[k].w)*>(kn + r * D));
          xv[k].w = __ldg(reinterpret_cast<const decltype(xv[k].w)*>(vn + r * D));
        } else {
          xk[k].w = decltype(xk[k].w){};
          xv[k].w = decltype(xv[k].w){};
        }
      }
#pragma unroll
      for (int k = 0; k < BATCH / 2; ++k) {
        const int r = r0 + k * RPW + sub;
        if (r0 + k * RPW >= hc) break;  // (the warp's)
        const int64_t off = __shfl_sync(FULL_MASK, dst, r & 31);
        const bool live = r < hc && off >= 0;
        float x0[4], x[4];
        xk[k].get(x0);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = x0[e];
        if (p.rotate_k) rotate<D, HALF>(x, tn.c, tn.s, l);
        if constexpr (Q4) {
          const Quad qk = quantise<D, HALF, true>(p, at, x0, x, l);
          if (live) store_quad<D>(p.k + off, qk, l);
          xv[k].get(x0);
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = x0[e];
          const Quad qv = quantise<D, HALF, false>(p, at, x0, x, l);
          if (live) store_quad<D>(p.v + off, qv, l);
        } else if (live) {
          if (p.rotate_k) xk[k].set(x);
          reinterpret_cast<decltype(xk[k].w)*>(p.k + off)[l] = xk[k].w;
          reinterpret_cast<decltype(xv[k].w)*>(p.v + off)[l] = xv[k].w;
        }
      }
    }
    if (p.q) {
      const int64_t q0 = static_cast<int64_t>(h0) * p.group * D + 4 * l;
      const T* q = static_cast<const T*>(p.q) + seq * p.q_seq + i * p.q_token + q0;
      T* qo = static_cast<T*>(p.q_out) + seq * p.qo_seq + i * p.qo_token + q0;
      const int rows = hc * p.group;
      for (int r0 = 0; r0 < rows; r0 += BATCH * RPW) {
        Raw<T> xq[BATCH];
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
          const int r = r0 + k * RPW + sub;
          xq[k].w = decltype(xq[k].w){};
          if (r < rows) xq[k].w = *reinterpret_cast<const decltype(xq[k].w)*>(q + r * D);  // (q_out may be q)
        }
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
          const int r = r0 + k * RPW + sub;
          float x[4];
          xq[k].get(x);
          rotate<D, HALF>(x, tn.c, tn.s, l);
          xq[k].set(x);
          if (r < rows) *reinterpret_cast<decltype(xq[k].w)*>(qo + r * D) = xq[k].w;
        }
      }
    }
  }
  if (p.token_tiles > 1) return;
  // this CTA has all tokens of its slices: their row counts, once every warp has read them
  __syncthreads();
  for (int j = threadIdx.x; j < head_ways * hpw && nn > 0; j += AW * 32) {
    const int h = ht * head_ways * hpw + j;
    if (h >= p.n_kv_heads) break;
    const int64_t s = append_slice(p, seq, h);
    const int n = p.n_valid[s];
    if (!rows_fit(p, n, nn)) continue;
    bool ok = true;
    if (p.rows.paged()) {
      const int32_t* trow = p.rows.seq_table(s);
      for (int k = n >> p.rows.block_shift; k <= (n + nn - 1) >> p.rows.block_shift; ++k) {
        const int blk = __ldg(trow + k);
        ok &= blk >= 0 && blk < p.rows.num_blocks;
      }
    }
    if (ok) p.n_valid[s] = n + nn;
  }
}

// Row counts of slices whose tokens several CTAs wrote: a warp per slice, after all of them.
__global__ void __launch_bounds__(AW * 32) append_count_kernel(const __grid_constant__ AppendParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int ls = blockIdx.x * AW + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int seq = ls / p.n_kv_heads, h = ls % p.n_kv_heads;
  if (seq >= p.n_seq) return;
  const int nn = append_tokens(p, seq);
  if (nn <= 0) return;
  const int64_t s = append_slice(p, seq, h);
  const int n = p.n_valid[s];
  if (!rows_fit(p, n, nn)) return;
  bool ok = true;
  if (p.rows.paged()) {
    const int32_t* trow = p.rows.seq_table(s);
    for (int k = (n >> p.rows.block_shift) + lane; k <= (n + nn - 1) >> p.rows.block_shift; k += 32) {
      const int blk = __ldg(trow + k);
      ok &= blk >= 0 && blk < p.rows.num_blocks;
    }
  }
  if (__all_sync(FULL_MASK, ok) && lane == 0) p.n_valid[s] = n + nn;
}

template <typename T, int D, bool Q4>
cudaError_t launch_style(const AppendParams& p, tri_rope_style style, cudaStream_t st) {
  auto kern = style == TRI_ROPE_HALF ? append_kernel<T, D, true, Q4> : append_kernel<T, D, false, Q4>;
  const int64_t ctas = static_cast<int64_t>(p.n_seq) * p.token_tiles * p.head_tiles;
  if (ctas > 0x7fffffff) return cudaErrorInvalidValue;
  kern<<<static_cast<unsigned>(ctas), AW * 32, 0, st>>>(p);
  note_launch();
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || p.token_tiles == 1) return e;
  cudaLaunchConfig_t cfg{};
  const int64_t slices = static_cast<int64_t>(p.n_seq) * p.n_kv_heads;
  cfg.gridDim = dim3(static_cast<unsigned>((slices + AW - 1) / AW));
  cfg.blockDim = dim3(AW * 32);
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, append_count_kernel, p);
  if (e == cudaSuccess) note_launch();
  return e;
}

// Launch shape. A warp's sines serve all of its heads, so it takes as many as leave enough warps to fill the
// GPU (152 SMs x 32). Few tokens per sequence go into one CTA, which then also advances the row counts;
// otherwise a second, early-launched kernel does.
void append_plan(AppendParams& p) {
  const int64_t tokens = static_cast<int64_t>(p.n_seq) * p.n_q, H = p.n_kv_heads;
  const int64_t hpw = std::max<int64_t>(1, std::min<int64_t>({tokens * H / (152 * 32), H, 32}));
  p.heads_per_warp = static_cast<int32_t>(hpw);
  int ways = 1;  // warps over heads
  while (ways < AW && ways * hpw < H) ways *= 2;
  if (p.n_q <= AW)
    while (AW / ways < p.n_q) ways /= 2;
  p.token_ways = AW / ways;
  p.token_tiles = (p.n_q + p.token_ways - 1) / p.token_ways;
  p.head_tiles = static_cast<int32_t>((H + ways * hpw - 1) / (ways * hpw));
}

}  // namespace

cudaError_t launch_append(AppendParams& p, tri_dtype dt, int head_dim, tri_rope_style style, cudaStream_t st) {
  append_plan(p);
  if (dt == TRI_Q4)
    return head_dim == 64 ? launch_style<__nv_bfloat16, 64, true>(p, style, st) : launch_style<__nv_bfloat16, 128, true>(p, style, st);
  if (dt == TRI_BF16)
    return head_dim == 64 ? launch_style<__nv_bfloat16, 64, false>(p, style, st) : launch_style<__nv_bfloat16, 128, false>(p, style, st);
  return head_dim == 64 ? launch_style<float, 64, false>(p, style, st) : launch_style<float, 128, false>(p, style, st);
}

}  // namespace tri
