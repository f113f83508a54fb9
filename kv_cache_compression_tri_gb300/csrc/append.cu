// append.cu -- new tokens into one layer of the cache, rotated on the way.
//
// Token i of a sequence becomes row n_valid + i of the layer's slices: V as it is,
// K (and the queries, into a buffer of their own) with band f multiplied by
// e^{i w_f p}. p is one of the token's positions, the one of the band's axis. The
// phase p w_f / 2 pi is a 64-bit fixed-point product, exact modulo a turn, so
// far positions keep their angle.
//
// Bound: every row is read once and written once, so HBM; instructions have to stay
// out of the way. A CTA takes a few tokens and a run of KV heads with their query heads.
// Its threads first compute the tokens' sines, one per band, into shared memory, and where
// each (token, head) row goes; then its warps take rows in groups. A lane has two
// chunks of eight elements, 8 l .. and d / 2 + 8 l .., so that a band's two elements are in one
// lane in either style, loads are 16 bytes, and a warp has four rows of d 128 or eight of
// d 64 (with four elements a lane and sines per warp, a 4-bit row took 270 instructions
// a warp and 8192 tokens 91 us). The next group's loads are in flight meanwhile.
//
// 4-bit rows: a quarter is four (two) lanes' chunks. Which fp16 or code is nearest is decided
// as in 64 bits: a lane bounds the error of its fp32 arithmetic, and where a border
// lies within it, the warp together repeats that quarter in fp64, an element a lane (about
// one of K in 500; a warp's fp64 instruction takes 16 clocks of an SM).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "attn_common.cuh"
#include "q4_common.cuh"

namespace tri {
namespace {

constexpr int AW = 4;  // warps per CTA (8192 tokens in 4 bits and read back: 58.6 us, with eight 60.8)
constexpr int MAX_HEADS = 16;  // KV heads of a CTA

// cos and sin of 2 pi frac(x nu): sincospi of the phase rounded to fp32 (within one step), and
// the first-order step for what the rounding left: error below 1.6 2^-24.
__device__ __forceinline__ float2 turn(int32_t x, uint64_t nu) {
  const int32_t hi = static_cast<int32_t>((static_cast<uint64_t>(static_cast<int64_t>(x)) * nu) >> 32);  // 2^-32 turns
  const float h = static_cast<float>(hi);
  const float rest = static_cast<float>(hi - static_cast<int32_t>(h)) * 1.4629180792671596e-09f;  // radians: 2 pi 2^-32
  float s, c;
  sincospif(h * 4.656612873077393e-10f, &s, &c);  // half turns: 2^-31
  return make_float2(fmaf(-s, rest, c), fmaf(c, rest, s));
}

// The band of entry i of pair k of lane l: what the lane's chunks need, in the order it is read.
template <int D, bool HALF>
__device__ __forceinline__ int band_of(int l, int k, int i) {
  return HALF ? 8 * l + 2 * k + i : (k < 2 ? 4 * l + 2 * k + i : D / 4 + 4 * l + 2 * (k - 2) + i);
}
__device__ __forceinline__ int axis_of(const AppendParams& p, int f) { return (p.axis_bits[f >> 4] >> (2 * (f & 15))) & 3; }

// n / d for n < 2^16 (magic: ceil(2^32 / d), 0 for d 1).
__device__ __forceinline__ int div_small(int n, uint32_t magic) { return magic ? static_cast<int>(__umulhi(n, magic)) : n; }

// A lane's two chunks of a row as loaded, a[0 .. 7] and b[0 .. 7].
template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  uint4 a, b;
  template <int D>
  __device__ __forceinline__ void load(const __nv_bfloat16* row, int l) {
    a = *reinterpret_cast<const uint4*>(row + 8 * l);
    b = *reinterpret_cast<const uint4*>(row + D / 2 + 8 * l);
  }
  template <int D>
  __device__ __forceinline__ void store(__nv_bfloat16* row, int l) const {
    *reinterpret_cast<uint4*>(row + 8 * l) = a;
    *reinterpret_cast<uint4*>(row + D / 2 + 8 * l) = b;
  }
  __device__ __forceinline__ static void unpack(uint4 w, float (&x)[8]) {
    x[0] = bf16_lo(w.x);
    x[1] = bf16_hi(w.x);
    x[2] = bf16_lo(w.y);
    x[3] = bf16_hi(w.y);
    x[4] = bf16_lo(w.z);
    x[5] = bf16_hi(w.z);
    x[6] = bf16_lo(w.w);
    x[7] = bf16_hi(w.w);
  }
  __device__ __forceinline__ void get(float (&x)[8], float (&y)[8]) const {
    unpack(a, x);
    unpack(b, y);
  }
  __device__ __forceinline__ void set(const float (&x)[8], const float (&y)[8]) {
    a = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
    b = make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
  }
};
template <>
struct Raw<float> {
  float4 w[4];
  template <int D>
  __device__ __forceinline__ void load(const float* row, int l) {
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = *reinterpret_cast<const float4*>(row + (k >> 1) * (D / 2) + 8 * l + 4 * (k & 1));
  }
  template <int D>
  __device__ __forceinline__ void store(float* row, int l) const {
#pragma unroll
    for (int k = 0; k < 4; ++k) *reinterpret_cast<float4*>(row + (k >> 1) * (D / 2) + 8 * l + 4 * (k & 1)) = w[k];
  }
  __device__ __forceinline__ void get(float (&x)[8], float (&y)[8]) const {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      x[4 * k] = w[k].x, x[4 * k + 1] = w[k].y, x[4 * k + 2] = w[k].z, x[4 * k + 3] = w[k].w;
      y[4 * k] = w[2 + k].x, y[4 * k + 1] = w[2 + k].y, y[4 * k + 2] = w[2 + k].z, y[4 * k + 3] = w[2 + k].w;
    }
  }
  __device__ __forceinline__ void set(const float (&x)[8], const float (&y)[8]) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      w[k] = make_float4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
      w[2 + k] = make_float4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
    }
  }
};

// The lane's chunks rotated; cs: the token's entries of this lane, pairs k LANES float4 apart.
template <int D, bool HALF>
__device__ __forceinline__ void rotate(float (&x)[8], float (&y)[8], const float4* cs) {
  constexpr int LANES = D / 16;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float4 t = cs[k * LANES];  // (cos, sin) of two bands
    if constexpr (HALF) {
      const float a0 = x[2 * k], b0 = y[2 * k], a1 = x[2 * k + 1], b1 = y[2 * k + 1];
      x[2 * k] = a0 * t.x - b0 * t.y;
      y[2 * k] = a0 * t.y + b0 * t.x;
      x[2 * k + 1] = a1 * t.z - b1 * t.w;
      y[2 * k + 1] = a1 * t.w + b1 * t.z;
    } else {
      float(&z)[8] = k < 2 ? x : y;
      const int e = 4 * (k & 1);
      const float a0 = z[e], b0 = z[e + 1], a1 = z[e + 2], b1 = z[e + 3];
      z[e] = a0 * t.x - b0 * t.y;
      z[e + 1] = a0 * t.y + b0 * t.x;
      z[e + 2] = a1 * t.z - b1 * t.w;
      z[e + 3] = a1 * t.w + b1 * t.z;
    }
  }
}

// A chunk's eight codes in order, and its quarter's (scale, minimum) as halves.
struct Chunk {
  uint32_t codes, pair;
};
__device__ __forceinline__ uint32_t pair_of(__half scale, __half low) {
  return __half_as_ushort(scale) | static_cast<uint32_t>(__half_as_ushort(low)) << 16;
}
constexpr uint32_t NAN_PAIR = 0x7fff7fffu;

// Quarter j of the row at `row`, in fp64, by the warp: an element a lane (d 64: lanes 16 .. 31 repeat). at:
// the token's positions, or NULL: not rotated. Chunk c of the quarter is returned to lane c's asker by `c`.
template <int D, bool HALF>
__device__ __noinline__ Chunk quarter64(const AppendParams& p, const __nv_bfloat16* row, const int32_t* at, int j, int c) {
  constexpr int QE = D / 4;
  const int i = (threadIdx.x & 31) % QE, e = j * QE + i;
  double x = static_cast<double>(__bfloat162float(row[e]));
  if (at) {
    const bool im = HALF ? e >= D / 2 : e & 1;
    const int f = HALF ? e % (D / 2) : e / 2;
    const double y = static_cast<double>(__bfloat162float(row[HALF ? e ^ (D / 2) : e ^ 1]));
    const int64_t t = static_cast<int64_t>(static_cast<uint64_t>(static_cast<int64_t>(__ldg(at + axis_of(p, f)))) * p.nu[f]);
    double cs, sn;
    sincospi(static_cast<double>(t) * 0x1p-63, &sn, &cs);
    x = im ? y * sn + x * cs : x * cs - y * sn;
  }
  constexpr double MOST = static_cast<double>(Q4_MOST);
  x = fmin(fmax(x, -MOST), MOST);
  // least and largest: by keys in the order of the numbers, in integers
  int64_t lo = __double_as_longlong(x);
  lo ^= static_cast<int64_t>(static_cast<uint64_t>(lo >> 63) >> 1);
  int64_t hi = lo;
#pragma unroll
  for (int k = QE / 2; k >= 1; k >>= 1) {
    const int64_t a = __shfl_xor_sync(FULL_MASK, lo, k), b = __shfl_xor_sync(FULL_MASK, hi, k);
    lo = a < lo ? a : lo;
    hi = b > hi ? b : hi;
  }
  auto number = [](int64_t key) { return __longlong_as_double(key ^ static_cast<int64_t>(static_cast<uint64_t>(key >> 63) >> 1)); };
  const __half low = __double2half(number(lo));
  const double m = static_cast<double>(__half2float(low));
  // scale and code: the nearest by fp32 reciprocals, then put right by exact comparisons with fifteen times the
  // midpoint to a neighbour, and with the scale times the middle of a step (ties to even)
  const double span = fmax(number(hi) - m, 0.0);
  uint32_t sb = __half_as_ushort(__float2half_rn(static_cast<float>(span) * (1.f / 15.f)));
  auto half_of = [](uint32_t bits) { return __half2float(__ushort_as_half(static_cast<unsigned short>(bits))); };
  const double above = static_cast<double>(7.5f * (half_of(sb) + half_of(sb + 1)));
  const double below = static_cast<double>(7.5f * (half_of(sb) + half_of(sb ? sb - 1 : 0)));
  if (span > above || (span == above && (sb & 1)))
    ++sb;
  else if (span < below || (span == below && (sb & 1)))
    --sb;
  const __half scale = __ushort_as_half(static_cast<unsigned short>(sb));
  const float s = __half2float(scale);
  const float whole = s > 0.f ? floorf(fminf(fmaxf(static_cast<float>(x - m) / s, 0.f), 15.f)) : 0.f;
  const double rest = (x - m) - static_cast<double>((whole + 0.5f) * s);
  uint32_t code = static_cast<uint32_t>(whole);
  if (s > 0.f && whole < 15.f && (rest > 0.0 || (rest == 0.0 && (code & 1)))) ++code;
  code <<= 4 * (i & 7);
#pragma unroll
  for (int k = 1; k <= 4; k <<= 1) code |= __shfl_xor_sync(FULL_MASK, code, k);
  return {__shfl_sync(FULL_MASK, code, 8 * c), pair_of(scale, low)};
}

// Minimum and maximum; a NaN makes NaN.
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b, float c) {
  float r;
  asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ uint32_t half_bits(float x) { return __half_as_ushort(__float2half_rn(x)); }

// Least and largest of a quarter, from this lane's chunk; a NaN in it makes both NaN.
template <int D>
__device__ __forceinline__ void bounds_of(const float (&x)[8], float& lo, float& hi) {
  lo = min_nan(min_nan(min_nan(x[0], x[1], x[2]), x[3], x[4]), min_nan(x[5], x[6], x[7]));
  hi = max_nan(max_nan(max_nan(x[0], x[1], x[2]), x[3], x[4]), max_nan(x[5], x[6], x[7]));
#pragma unroll
  for (int k = 1; k < D / 32; k <<= 1) {
    lo = min_nan(lo, __shfl_xor_sync(FULL_MASK, lo, k));
    hi = max_nan(hi, __shfl_xor_sync(FULL_MASK, hi, k));
  }
}
__device__ __forceinline__ float limit(float x) { return max_nan(min_nan(x, Q4_MOST), -Q4_MOST); }

// A chunk in fp32; err: how far its elements, and lo and hi, may be off. border: some decision may
// differ from fp64's.
__device__ __forceinline__ Chunk quantise(const float (&x)[8], float lo, float hi, float err, bool& border) {
  const __half low = __float2half_rn(lo);
  const float m = __half2float(low), span = fmaxf(hi - m, 0.f);
  border = half_bits(lo - err) != half_bits(lo + err);
  // scale: fifteen times the midpoints to its neighbours (16 bits: exact) against the span, which errs by its rounding
  const __half scale = __float2half_rn(span * (1.f / 15.f));
  const float s = __half2float(scale), es = fmaf(span, 0x1p-24f, err);
  const uint32_t sb = __half_as_ushort(scale);
  const float up = __half2float(__ushort_as_half(static_cast<unsigned short>(sb + 1)));
  const float down = __half2float(__ushort_as_half(static_cast<unsigned short>(sb ? sb - 1 : 0)));
  border |= span + es >= 7.5f * (s + up) || span - es < 7.5f * (s + down);
  // codes: v = u / 15 within 0 .. 1; u errs by the elements' error over the scale, 2^-21 of the largest element over
  // the scale for the reciprocal and the products, and 2^-19
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
  inv = s > 0.f ? inv : 0.f;
  const float near = 0.5f - fmaf(fmaf(fmaxf(fabsf(lo), fabsf(hi)), 0x1p-21f, err), inv, 0x1p-19f);
  const float inv15 = inv * (1.f / 15.f), b = -m * inv15;
  constexpr float MAGIC = 12582912.f;  // 1.5 2^23: adding it rounds to a whole number, ties to even
  float far = 0.f, c[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float v = __saturatef(fmaf(x[e], inv15, b));  // (NaN: 0)
    c[e] = fmaf(v, 15.f, MAGIC) - MAGIC;
    far = fmaxf(far, fabsf(fmaf(v, 15.f, -c[e])));
  }
  border |= far > near;
  const float p0 = fmaf(fmaf(fmaf(c[3], 16.f, c[2]), 16.f, c[1]), 16.f, c[0]) + 8388608.f;  // low 16 bits: four codes
  const float p1 = fmaf(fmaf(fmaf(c[7], 16.f, c[6]), 16.f, c[5]), 16.f, c[4]) + 8388608.f;
  const bool nan = lo != lo;
  border &= !nan;
  return {nan ? 0u : __byte_perm(__float_as_uint(p0), __float_as_uint(p1), 0x5410), nan ? NAN_PAIR : pair_of(scale, low)};
}

// A lane's chunks a and b of a row, to the 4-bit row at `row` (live: it is there).
template <int D>
__device__ __forceinline__ void store_chunks(char* row, bool live, const Chunk& a, const Chunk& b, int l) {
  constexpr int QL = D / 32;  // lanes of a quarter: chunk a is of quarter l / QL, b of the one two on
  uint2 w;
  int at;
  if constexpr (D == 128) {
    // lanes t and t + 4 hold words 4 t + (0, 2) and 4 t + (1, 3)
    const uint32_t other = __shfl_xor_sync(FULL_MASK, l < 4 ? b.codes : a.codes, 4);
    w = l < 4 ? make_uint2(a.codes, other) : make_uint2(other, b.codes);
    at = 4 * (l & 3) + (l < 4 ? 0 : 2);
  } else {
    // a word has four codes of quarter 2 k in bytes 0 and 2 and of 2 k + 1 in bytes 1 and 3: lanes l and l + 2
    const uint32_t a2 = __shfl_xor_sync(FULL_MASK, a.codes, 2), b2 = __shfl_xor_sync(FULL_MASK, b.codes, 2);
    w = l < 2 ? make_uint2(__byte_perm(a.codes, a2, 0x5140), __byte_perm(b.codes, b2, 0x5140))
              : make_uint2(__byte_perm(a2, a.codes, 0x7362), __byte_perm(b2, b.codes, 0x7362));
    at = 2 * (2 * (l & 1) + (l >> 1));
  }
  if (!live) return;
  *reinterpret_cast<uint2*>(row + 4 * at) = w;
  if (l % QL == 0) {
    uint32_t* pairs = reinterpret_cast<uint32_t*>(row + Q4Row<D>::CODES);
    pairs[l / QL] = a.pair;
    pairs[l / QL + 2] = b.pair;
  }
}

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

// A lane's chunks of a row, as 4-bit codes to `to` (live: it is there). src: the row as it came (NULL: none); at: the
// token's positions if x and y are rotated.
template <int D, bool HALF>
__device__ __forceinline__ void store_q4(const AppendParams& p, char* to, bool live, const float (&x)[8], const float (&y)[8],
                                         const __nv_bfloat16* src, const int32_t* at, int l, int lane) {
  constexpr int QL = D / 32;  // lanes of a quarter
  float la, ha, lb, hb;
  bounds_of<D>(x, la, ha);
  bounds_of<D>(y, lb, hb);
  // a rotated element errs by at most 1.4 2^-22 of its larger input, which is at most sqrt(2) of the larger
  // of the rotated pair; a pair in halves has one in each quarter
  float ma = fmaxf(fabsf(la), fabsf(ha)), mb = fmaxf(fabsf(lb), fabsf(hb));
  if (HALF) ma = mb = fmaxf(ma, mb);
  const float ea = at ? ma * 0x1p-21f : 0.f, eb = at ? mb * 0x1p-21f : 0.f;
  bool border_a, border_b;
  Chunk a = quantise(x, limit(la), limit(ha), ea, border_a), b = quantise(y, limit(lb), limit(hb), eb, border_b);
  if (__any_sync(FULL_MASK, (border_a || border_b) && src)) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      unsigned todo = __ballot_sync(FULL_MASK, (k ? border_b : border_a) && src);
      while (todo) {
        // the first of a quarter's lanes asks; all of them take
        const int asks = (__ffs(todo) - 1) / QL * QL;
        todo &= ~(((1u << QL) - 1) << asks);
        const auto row = reinterpret_cast<const __nv_bfloat16*>(__shfl_sync(FULL_MASK, reinterpret_cast<uintptr_t>(src), asks));
        const auto pos = reinterpret_cast<const int32_t*>(__shfl_sync(FULL_MASK, reinterpret_cast<uintptr_t>(at), asks));
        const int quarter = __shfl_sync(FULL_MASK, l / QL + 2 * k, asks);
        const Chunk e = quarter64<D, HALF>(p, row, pos, quarter, lane % QL);
        if (lane / QL * QL == asks) (k ? b : a) = e;
      }
    }
  }
  store_chunks<D>(to, live, a, b, l);
}

// Rows (token, head) of `toks` tokens in steps of AW groups of RPW from group g on, the next one's loads in flight:
// f(whether there is a row, token, head, source, its chunks), by whole warps. `per`: heads of a token in
// the numbering, `live` of them there; magic and step (AW groups as tokens and heads) belong to `per`.
// first: the chunks of group g's row, from first_row.
template <typename T, int D>
__device__ __forceinline__ Raw<T> first_row(const T* base, int64_t token, int toks, int per, int live, uint32_t magic, int g, int sub, int l) {
  const int n = g * (32 / (D / 16)) + sub, tok = div_small(n, magic), head = n - tok * per;
  Raw<T> r{};
  if (n < toks * per && head < live) r.template load<D>(base + tok * token + head * D, l);
  return r;
}
template <typename T, int D, class Fn>
__device__ __forceinline__ void for_rows(const T* base, int64_t token, int toks, int per, int live, uint32_t magic, int2 step, int g, int sub,
                                         int l, const Raw<T>& first, Fn f) {
  constexpr int RPW = 32 / (D / 16);
  int n = g * RPW, tok = div_small(n + sub, magic), head = n + sub - tok * per;
  const T* src = base + tok * token + head * D;
  const int rows = toks * per;
  Raw<T> next = first;
  bool in = n + sub < rows && head < live;
  while (n < rows) {
    Raw<T> cur = next;
    const bool in_now = in;
    const int tok_now = in ? tok : 0, head_now = head;
    const T* src_now = src;
    n += AW * RPW;
    tok += step.x;
    head += step.y;
    src += step.x * token + step.y * D;
    if (head >= per) {
      head -= per;
      ++tok;
      src += token - per * D;
    }
    in = n + sub < rows && head < live;
    if (in) next.template load<D>(src, l);
    f(in_now, tok_now, head_now, src_now, cur);
  }
}

template <typename T, int D, bool HALF, bool Q4>
__global__ void __launch_bounds__(AW * 32, 8) append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int LANES = D / 16, RPW = 32 / LANES, F = D / 2;  // lanes of a row, rows of a warp
  constexpr int MAX_TOKENS = AW * 32 / F;
  __shared__ float4 turns[MAX_TOKENS][F / 2];
  static_assert(MAX_TOKENS * MAX_HEADS <= AW * 32, "a thread per row");
  __shared__ int64_t dst[MAX_TOKENS * MAX_HEADS];  // byte offset of each (token, head) row in K and V, -1: none
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int t = threadIdx.x, w = t >> 5, lane = t & 31, sub = lane / LANES, l = lane % LANES;
  int b = blockIdx.x;
  const int ht = b % p.head_tiles;
  b /= p.head_tiles;
  const int tt = b % p.token_tiles, seq = b / p.token_tiles;
  const int H = p.heads, h0 = ht * H, hc = min(H, p.n_kv_heads - h0), i0 = tt * p.tokens;
  const int nn = append_tokens(p, seq), toks = min(p.tokens, nn - i0);
  const int32_t* positions = p.positions + (static_cast<int64_t>(seq) * p.n_q + i0) * p.n_axes;
  if (toks > 0) {
    // Rows (token, head) in groups of RPW, a warp's groups AW apart: first those of K, then of V, then of the queries,
    // whose first groups go to the warps behind the last of the kind before.
    const int kv_groups = (toks * H + RPW - 1) / RPW;
    const T* kn = static_cast<const T*>(p.kn) + seq * p.k_seq + i0 * p.k_token + static_cast<int64_t>(h0) * D;
    const T* vn = static_cast<const T*>(p.vn) + seq * p.v_seq + i0 * p.v_token + static_cast<int64_t>(h0) * D;
    const int64_t q0 = static_cast<int64_t>(h0) * p.group * D;
    const T* q = static_cast<const T*>(p.q) + seq * p.q_seq + i0 * p.q_token + q0;
    const int vg = (w - kv_groups) & (AW - 1), qg = (w - 2 * kv_groups) & (AW - 1);
    // (their loads are on the way while the sines are computed)
    const Raw<T> k_first = first_row<T, D>(kn, p.k_token, toks, H, hc, p.head_magic, w, sub, l);
    const Raw<T> v_first = first_row<T, D>(vn, p.v_token, toks, H, hc, p.head_magic, vg, sub, l);
    const Raw<T> q_first = first_row<T, D>(q, p.q_token, toks, H * p.group, hc * p.group, p.q_magic, qg, sub, l);
    if (t < toks * F) {
      const int tok = t / F, e = t % F, k = e / (2 * LANES), lk = e / 2 % LANES;
      const int f = band_of<D, HALF>(lk, k, e & 1);
      reinterpret_cast<float2*>(turns[tok])[e] = turn(__ldg(positions + tok * p.n_axes + axis_of(p, f)), p.nu[f]);
    }
    if (t < toks * H) {
      const int tok = div_small(t, p.head_magic), h = t - tok * H;
      int64_t to = -1;
      if (h < hc) {
        const int64_t s = append_slice(p, seq, h0 + h);
        const int n = p.n_valid[s];
        if (rows_fit(p, n, nn)) {
          const int row = n + i0 + tok;
          bool ok = true;
          int64_t at = s * p.rows.slice_bytes + static_cast<int64_t>(row) * p.rows.row_bytes;
          if (p.rows.paged()) {
            const int blk = __ldg(p.rows.table + static_cast<int64_t>(seq) * p.rows.max_blocks + (row >> p.rows.block_shift));
            ok = blk >= 0 && blk < p.rows.num_blocks;
            if (!ok) set_status(p.dev_status, TRI_DEV_BAD_BLOCK);
            at = blk * p.rows.block_bytes + p.layer * p.rows.layer_bytes + (h0 + h) * p.rows.head_bytes +
                 (row & (p.rows.block_size - 1)) * p.rows.row_bytes;
          }
          if (ok) {
            to = at;
            if (p.pos) p.pos[s * p.n_cap + row] = __ldg(positions + tok * p.n_axes);
          }
        }
      }
      dst[t] = to;
    }
    __syncthreads();
    for_rows<T, D>(kn, p.k_token, toks, H, hc, p.head_magic, p.head_step, w, sub, l, k_first, [&](bool in, int tok, int head, const T* src, Raw<T>& cur) {
      const float4* cs = turns[tok] + l;
      const int64_t off = in ? dst[tok * H + head] : -1;
      char* to = p.k + (off >= 0 ? off : 0);
      if constexpr (Q4) {
        float x[8], y[8];
        cur.get(x, y);
        if (p.rotate_k) rotate<D, HALF>(x, y, cs);
        store_q4<D, HALF>(p, to, off >= 0, x, y, in ? reinterpret_cast<const __nv_bfloat16*>(src) : nullptr,
                          p.rotate_k ? positions + tok * p.n_axes : nullptr, l, lane);
      } else {
        if (p.rotate_k) {
          float x[8], y[8];
          cur.get(x, y);
          rotate<D, HALF>(x, y, cs);
          cur.set(x, y);
        }
        if (off >= 0) cur.template store<D>(reinterpret_cast<T*>(to), l);
      }
    });
    for_rows<T, D>(vn, p.v_token, toks, H, hc, p.head_magic, p.head_step, vg, sub, l, v_first,
                   [&](bool in, int tok, int head, const T* src, Raw<T>& cur) {
      const int64_t off = in ? dst[tok * H + head] : -1;
      char* to = p.v + (off >= 0 ? off : 0);
      if constexpr (Q4) {
        float x[8], y[8];
        cur.get(x, y);
        store_q4<D, HALF>(p, to, off >= 0, x, y, in ? reinterpret_cast<const __nv_bfloat16*>(src) : nullptr, nullptr, l, lane);
      } else {
        if (off >= 0) cur.template store<D>(reinterpret_cast<T*>(to), l);
      }
    });
    if (p.q) {
      T* qo = static_cast<T*>(p.q_out) + seq * p.qo_seq + i0 * p.qo_token + q0;
      for_rows<T, D>(q, p.q_token, toks, H * p.group, hc * p.group, p.q_magic, p.q_step, qg, sub, l, q_first,
                     [&](bool in, int tok, int head, const T*, Raw<T>& cur) {
        float x[8], y[8];
        cur.get(x, y);
        rotate<D, HALF>(x, y, turns[tok] + l);
        cur.set(x, y);
        if (in) cur.template store<D>(qo + tok * p.qo_token + head * D, l);
      });
    }
  }
  if (p.token_tiles > 1) return;
  // this CTA has all tokens of its slices: their row counts, once every thread has read them
  __syncthreads();
  if (t < hc && nn > 0) {
    const int64_t s = append_slice(p, seq, h0 + t);
    const int n = p.n_valid[s];
    if (!rows_fit(p, n, nn)) return;
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
  if (ctas > 0x7fffffff) return cudaErrorNotSupported;  // (more than a launch counts)
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

uint32_t magic_of(int d) { return d == 1 ? 0u : static_cast<uint32_t>(((uint64_t{1} << 32) + d - 1) / d); }

// Launch shape: the tokens of a CTA are at most one per sine that its threads compute in one go, and fewer where
// that would leave SMs without a CTA. A sequence's tokens that fit one CTA go there, which then also
// advances the row counts; otherwise a second, early-launched kernel does.
void append_plan(AppendParams& p, int head_dim) {
  const int64_t tokens = static_cast<int64_t>(p.n_seq) * p.n_q;
  const int most = AW * 32 / (head_dim / 2);
  p.heads = std::min(p.n_kv_heads, MAX_HEADS);
  p.head_tiles = (p.n_kv_heads + p.heads - 1) / p.heads;
  p.tokens = p.n_q <= most ? p.n_q : static_cast<int32_t>(std::max<int64_t>(1, std::min<int64_t>(most, tokens * p.head_tiles / (2 * 152))));
  p.token_tiles = (p.n_q + p.tokens - 1) / p.tokens;
  p.head_magic = magic_of(p.heads);
  const int per = p.heads * std::max(p.group, 1), step = AW * 32 / (head_dim / 16);
  p.q_magic = magic_of(per);
  p.head_step = make_int2(step / p.heads, step % p.heads);
  p.q_step = make_int2(step / per, step % per);
}

}  // namespace

cudaError_t launch_append(AppendParams& p, tri_dtype dt, int head_dim, tri_rope_style style, cudaStream_t st) {
  append_plan(p, head_dim);
  if (dt == TRI_Q4)
    return head_dim == 64 ? launch_style<__nv_bfloat16, 64, true>(p, style, st) : launch_style<__nv_bfloat16, 128, true>(p, style, st);
  if (dt == TRI_BF16)
    return head_dim == 64 ? launch_style<__nv_bfloat16, 64, false>(p, style, st) : launch_style<__nv_bfloat16, 128, false>(p, style, st);
  return head_dim == 64 ? launch_style<float, 64, false>(p, style, st) : launch_style<float, 128, false>(p, style, st);
}

}  // namespace tri
