// Quantise new keys and values into the pages of an 8-bit cache.
//
// A unit of work is one (sequence, page it touches, head) for keys or for
// values: the scale belongs to the page and head, so the unit's new elements
// are read once into registers, their largest magnitude is reduced over the
// CTA, and the same registers are then rounded to e4m3 and stored. The new
// scale is a power of two, so x / s' is exact (a change of exponent) and the
// only rounding is the one to e4m3; codes that were in the page before are read
// and stored again only when the scale grows.
//
// Bound by latency for the decode step (a few hundred bytes a unit: 3 us in a
// graph for 64 tokens of 8 heads) and by HBM for prompts (2 bytes read, 1 written
// an element): 191 MB in 30.3 us, 6.3 TB/s. What counts there is the instructions
// an element. Magnitudes are compared as packed 16-bit integers and the product
// with the power of two is taken in packed bf16; what is rare (infinities and NaN
// that must not set the scale, an old scale that is no power of two) reads its
// elements again in loops of its own. Filtering every element and dividing in the
// main loop took 38.9 us, with every issue slot but a third busy.
#include "kv8_device.cuh"
#include "w4a16_device.cuh"

namespace w4 {
namespace kv8 {
namespace {

constexpr int AT = 128;  // threads of a unit

struct Append {
  const uint16_t *k, *v;
  size_t k_stride, v_stride;
  Cache c;
  const int32_t *table, *kv_lens, *cu_q;
  int table_stride, batch, total_q, max_q, pages_per_seq;
  int* status;
};

// The smallest exponent n >= -40 with amax <= 448 * 2^n: amax = m 2^e with m in
// [0.5, 1) and 448 = 0.875 * 2^9, so n = e - 9, one more when m > 0.875.
__device__ __forceinline__ int fit_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int n = (int)(u >> 23) - 126 - 9 + ((u & 0x7FFFFFu) > 0x600000u);
  return max(n, -40);
}
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

template <bool BF16>
__device__ __forceinline__ float2 unpack(uint32_t w) {
  if constexpr (BF16)
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  else
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// The largest of eight magnitudes and m, by halves: as bits they order as numbers do.
__device__ __forceinline__ uint32_t max_abs(uint32_t m, const uint4& x) {
  constexpr uint32_t MAG = 0x7FFF7FFFu;
  return __vmaxu2(__vmaxu2(__vmaxu2(m, x.x & MAG), x.y & MAG), __vmaxu2(x.z & MAG, x.w & MAG));
}

// Four codes of x / s for s a power of two (inv = 1 / s as a bf16 pair, or fp32).
// In bf16 the product is exact, or below half the smallest code and rounds to 0.
template <bool BF16>
__device__ __forceinline__ uint32_t codes4(uint32_t w0, uint32_t w1, float inv, uint32_t inv2) {
  float2 f0, f1;
  if constexpr (BF16) {
    f0 = unpack<true>(mul_x2<true>(w0, inv2));
    f1 = unpack<true>(mul_x2<true>(w1, inv2));
  } else {
    f0 = unpack<false>(w0);
    f1 = unpack<false>(w1);
    f0 = make_float2(f0.x * inv, f0.y * inv);
    f1 = make_float2(f1.x * inv, f1.y * inv);
  }
  return (uint32_t)f32x2_to_e4m3x2(f0.x, f0.y) | (uint32_t)f32x2_to_e4m3x2(f1.x, f1.y) << 16;
}

// NV: 16-byte pieces of new elements a thread may hold (a page of one head has
// page * D / 8 of them).
template <int D, int NV, bool BF16>
__global__ void __launch_bounds__(AT) append_kernel(const Append a) {
  grid_wait();
  grid_launch_dependents();
  const int b = blockIdx.x / a.pages_per_seq;
  const int idx = blockIdx.x - b * a.pages_per_seq;
  const int h = blockIdx.y >> 1;
  const bool is_v = blockIdx.y & 1;
  const int q0 = a.cu_q[b], n = a.cu_q[b + 1] - q0, kv = a.kv_lens[b];
  const int shift = a.c.page_shift;
  if (n == 0 && q0 >= 0) return;
  if (q0 < 0 || n < 0 || n > a.max_q || q0 > a.total_q - n || n > kv || kv > MAX_KV ||
      kv > ((long long)a.table_stride << shift)) {
    if (threadIdx.x == 0) record(a.status, W4_ERR_PAGE);
    return;
  }
  const int first = kv - n;                      // the first new token
  const int pi = (first >> shift) + idx;         // page of the sequence
  const int lo = max(first, pi << shift), hi = min(kv, (pi + 1) << shift);
  if (lo >= hi) return;
  const int p = a.table[(size_t)b * a.table_stride + pi];  // (looked at after the elements are on their way)
  constexpr int RP = D / 8;  // 16-byte pieces of a row
  const int pieces = (hi - lo) * RP;
  const size_t stride = is_v ? a.v_stride : a.k_stride;
  const uint16_t* src = (is_v ? a.v : a.k) + (size_t)(q0 + lo - first) * stride + (size_t)h * D;
  const uint16_t* mine = src + (threadIdx.x / RP) * stride + (threadIdx.x % RP) * 8;
  uint4 x[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    x[j] = make_uint4(0, 0, 0, 0);
    if (threadIdx.x + j * AT < pieces)
      x[j] = *reinterpret_cast<const uint4*>(mine + j * (AT / RP) * stride);
  }
  if (p < 0 || p >= a.c.pages) {
    if (threadIdx.x == 0) record(a.status, W4_ERR_PAGE);
    return;
  }
  const size_t ph = (size_t)p * a.c.heads + h;
  float* scale = (is_v ? a.c.vs : a.c.ks) + ph;
  const int held = lo - (pi << shift);  // this sequence's tokens already in the page
  const float old = held > 0 ? *scale : 0.f;
  constexpr uint32_t INF = BF16 ? 0x7F80u : 0x7C00u;
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < NV; ++j) m = max_abs(m, x[j]);
  m = max(m & 0xFFFFu, m >> 16);
  if (m >= INF) {  // infinities and NaN do not set the scale: look again, without them
    m = 0;
    for (int i = threadIdx.x; i < pieces; i += AT)
      for (int k = 0; k < 8; ++k) {
        const uint32_t u = src[(size_t)(i / RP) * stride + (i % RP) * 8 + k] & 0x7FFFu;
        if (u < INF) m = max(m, u);
      }
  }
  m = __reduce_max_sync(~0u, m);
  __shared__ uint32_t red[AT / 32];
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < AT / 32; ++i) m = max(m, red[i]);
  const float amax = half_bits_to_float<BF16>((uint16_t)m);
  const int e = fit_exponent(amax);
  const float fit = pow2f(e);
  const bool grows = !(old >= fit);
  const float now = grows ? fit : old;
  // the new scale is a power of two unless an old one of another kind stays
  const float inv = grows ? pow2f(-e) : __fdiv_rn(1.f, now);
  const bool exact_inv = (__float_as_uint(now) & 0x7FFFFFu) == 0;
  uint8_t* codes = (is_v ? a.c.v : a.c.k) + ((ph << shift) * D);
  if (held > 0 && grows) {
    const float ratio = __fdiv_rn(old, now);
    uint4* o = reinterpret_cast<uint4*>(codes);
    for (int i = threadIdx.x; i < held * (D / 16); i += AT) {
      uint4 c = o[i];
      uint32_t* w = reinterpret_cast<uint32_t*>(&c);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t lo2 = e4m3x2_to_f16x2((uint16_t)(w[j] & 0xFFFF));
        uint32_t hi2 = e4m3x2_to_f16x2((uint16_t)(w[j] >> 16));
        const float2 f0 = __half22float2(*reinterpret_cast<__half2*>(&lo2));
        const float2 f1 = __half22float2(*reinterpret_cast<__half2*>(&hi2));
        w[j] = (uint32_t)f32x2_to_e4m3x2(f0.x * ratio, f0.y * ratio) |
               ((uint32_t)f32x2_to_e4m3x2(f1.x * ratio, f1.y * ratio) << 16);
      }
      o[i] = c;
    }
  }
  uint8_t* to = codes + (size_t)held * D;
  if (exact_inv) {
    const uint32_t inv2 = (__float_as_uint(inv) >> 16) * 0x10001u;
    uint8_t* to0 = to + threadIdx.x * 8;
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (threadIdx.x + j * AT < pieces)
        *reinterpret_cast<uint2*>(to0 + j * AT * 8) =
            make_uint2(codes4<BF16>(x[j].x, x[j].y, inv, inv2), codes4<BF16>(x[j].z, x[j].w, inv, inv2));
  } else {  // an old scale of another kind stays
    for (int i = threadIdx.x; i < pieces; i += AT)
      for (int k = 0; k < 8; k += 2) {
        const float2 f = unpack<BF16>(*reinterpret_cast<const uint32_t*>(
            src + (size_t)(i / RP) * stride + (i % RP) * 8 + k));
        *reinterpret_cast<uint16_t*>(to + (size_t)i * 8 + k) =
            f32x2_to_e4m3x2(__fdiv_rn(f.x, now), __fdiv_rn(f.y, now));
      }
  }
  if (threadIdx.x == 0) *scale = now;
}

template <int D, bool BF16>
cudaError_t launch_d(const Append& a, dim3 grid, cudaStream_t s) {
  // pieces of 16 bytes a thread: up to a page of new tokens, or all a sequence has
  const int rows = min(1 << a.c.page_shift, a.max_q);
  const int nv = (rows * (D / 8) + AT - 1) / AT;
  if (nv <= 1) return launch(append_kernel<D, 1, BF16>, grid, AT, 0, s, a);
  if (nv <= 2) return launch(append_kernel<D, 2, BF16>, grid, AT, 0, s, a);
  if (nv <= 4) return launch(append_kernel<D, 4, BF16>, grid, AT, 0, s, a);
  if (nv <= 8) return launch(append_kernel<D, 8, BF16>, grid, AT, 0, s, a);
  return launch(append_kernel<D, 16, BF16>, grid, AT, 0, s, a);
}

}  // namespace

cudaError_t launch_append(const AppendArgs& a, cudaStream_t s) {
  int* status = nullptr;
  const cudaError_t e = device_status_ptr(&status);
  if (e != cudaSuccess) return e;
  const int page = 1 << a.c.page_shift;
  const int per = (a.max_q + page - 2) / page + 1;  // pages n tokens can touch
  if ((long long)per * a.batch >= (1ll << 31)) return cudaErrorInvalidValue;
  const Append p{a.k, a.v, a.k_stride, a.v_stride, a.c, a.table, a.kv_lens, a.cu_q,
                 a.table_stride, a.batch, a.total_q, a.max_q, per, status};
  const dim3 grid(per * a.batch, 2 * a.c.heads);
  if (a.dim == 64) return a.bf16 ? launch_d<64, true>(p, grid, s) : launch_d<64, false>(p, grid, s);
  return a.bf16 ? launch_d<128, true>(p, grid, s) : launch_d<128, false>(p, grid, s);
}

}  // namespace kv8
}  // namespace w4
