// Keep the accepted drafts of a checked tree in an 8-bit cache.
//
// Of a sequence's n drafts (its last n tokens) those that path lists move together:
// draft path[i] becomes the sequence's i-th new token. path ascends, so what moves is
// path[f..m) for the first f with path[f] != f, every move is towards the front, and
// only the first page that gets tokens can hold others that stay: those before draft f.
//
// Codes share their page's scale, so a page that gets tokens from louder pages takes
// their scale, s' = max(s of the sources, and its own if tokens stay in it), and codes
// are stored again as e4m3(code * (s / s')), in fp32; with the powers of two that
// w4_kv8_append makes that changes only the exponent.
//
// A CTA has the keys or the values of one sequence and head: it reads all that moves
// into registers before it writes any of it. Bound by latency: bounds, path and page
// numbers, scales and codes are three reads that follow one another. 2.5 us for one
// sequence's 27 of 61 drafts, 3.4 us for 64 sequences (8 kv heads of 128, in a graph).
#include "kv8_device.cuh"

namespace w4 {
namespace kv8 {
namespace {

constexpr int KT = 128;                      // threads
constexpr int SPAN = MAX_DRAFTS / 16 + 1;    // pages that the drafts can touch

struct Keep {
  Cache c;
  const int32_t *table, *kv_lens, *cu_q, *path;
  int table_stride, total_q, max_q;
  int* status;
};

// Sixteen codes times r (at most 1).
__device__ __forceinline__ uint4 times(uint4 x, float r) {
  uint32_t* w = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t lo = e4m3x2_to_f16x2((uint16_t)(w[j] & 0xFFFF)), hi = e4m3x2_to_f16x2((uint16_t)(w[j] >> 16));
    const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    w[j] = (uint32_t)f32x2_to_e4m3x2(f0.x * r, f0.y * r) | (uint32_t)f32x2_to_e4m3x2(f1.x * r, f1.y * r) << 16;
  }
  return x;
}

template <int D>
__global__ void __launch_bounds__(KT) keep_kernel(const Keep k) {
  constexpr int RP = D / 16;                 // 16-byte pieces of a token
  constexpr int NV = MAX_DRAFTS * RP / KT;   // that a thread may hold
  __shared__ int path_sh[MAX_DRAFTS], first_sh, count_sh, row_sh[SPAN], now_sh[SPAN];
  __shared__ float scale_sh[SPAN];
  grid_wait();
  grid_launch_dependents();
  const int b = blockIdx.x, h = blockIdx.y >> 1, tid = threadIdx.x;
  const bool is_v = blockIdx.y & 1;
  const int q0 = k.cu_q[b], n = k.cu_q[b + 1] - q0, kv = k.kv_lens[b], shift = k.c.page_shift;
  if (n == 0 && q0 >= 0) return;
  if (q0 < 0 || n < 0 || n > k.max_q || q0 > k.total_q - n || n > kv || kv > MAX_KV ||
      kv > ((long long)k.table_stride << shift)) {
    if (tid == 0 && blockIdx.y == 0) record(k.status, W4_ERR_PAGE);
    return;
  }
  const int base = kv - n, page0 = base >> shift, pages = ((kv - 1) >> shift) - page0 + 1;
  const int mine = tid < n ? k.path[q0 + tid] : -1;
  const int page = tid < pages ? k.table[(size_t)b * k.table_stride + page0 + tid] : 0;
  if (tid < MAX_DRAFTS) path_sh[tid] = mine;
  if (tid == 0) first_sh = count_sh = 0;
  if (tid < SPAN) now_sh[tid] = 0;
  __syncthreads();
  // what is listed ascends and lies among the drafts; behind it there is nothing
  const int last = tid > 0 && tid < MAX_DRAFTS ? path_sh[tid - 1] : -1;
  const bool listed = mine >= 0;
  bool bad = listed && (mine >= n || mine <= last || (tid > 0 && last < 0));
  bad = bad || page < 0 || page >= k.c.pages;
  if (listed) atomicAdd(&count_sh, 1);
  if (listed && mine == tid) atomicAdd(&first_sh, 1);  // (a prefix: it ascends)
  if (__syncthreads_or(bad)) {
    if (tid == 0 && blockIdx.y == 0) record(k.status, W4_ERR_PAGE);
    return;
  }
  const int first = first_sh, count = count_sh;
  if (first == count) return;  // nothing moves
  float* scales = is_v ? k.c.vs : k.c.ks;
  uint8_t* codes = is_v ? k.c.v : k.c.k;
  if (tid < pages) {
    row_sh[tid] = page * k.c.heads + h;
    scale_sh[tid] = scales[(size_t)page * k.c.heads + h];
  }
  __syncthreads();
  const int mask = (1 << shift) - 1;
  auto at = [&](int j) {  // token j's codes
    return codes + (((size_t)row_sh[(j >> shift) - page0] << shift) + (j & mask)) * D;
  };
  uint4 x[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int i = first + (tid + v * KT) / RP;
    if (i < count) x[v] = *reinterpret_cast<const uint4*>(at(base + path_sh[i]) + 16 * (tid % RP));
  }
  const int to0 = base + first, held = to0 & mask;  // held: tokens that stay in the first page
  if (tid >= first && tid < count)  // (scales are positive, so their bits order as they do)
    atomicMax(&now_sh[((base + tid) >> shift) - page0], __float_as_int(scale_sh[((base + mine) >> shift) - page0]));
  const int p0 = (to0 >> shift) - page0;
  if (tid == 0 && held > 0) atomicMax(&now_sh[p0], __float_as_int(scale_sh[p0]));
  __syncthreads();
  const float old = scale_sh[p0], grown = __int_as_float(now_sh[p0]);
  if (held > 0 && grown != old) {
    const float r = __fdiv_rn(old, grown);
    uint4* o = reinterpret_cast<uint4*>(codes + ((size_t)row_sh[p0] << shift) * D);
    for (int i = tid; i < held * RP; i += KT) o[i] = times(o[i], r);
  }
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int i = first + (tid + v * KT) / RP;
    if (i >= count) continue;
    const float s = scale_sh[((base + path_sh[i]) >> shift) - page0];
    const float now = __int_as_float(now_sh[((base + i) >> shift) - page0]);
    *reinterpret_cast<uint4*>(at(base + i) + 16 * (tid % RP)) = s == now ? x[v] : times(x[v], __fdiv_rn(s, now));
  }
  if (tid >= p0 && tid <= ((base + count - 1) >> shift) - page0) scales[row_sh[tid]] = __int_as_float(now_sh[tid]);
}

}  // namespace

cudaError_t launch_keep(const KeepArgs& a, cudaStream_t s) {
  int* status = nullptr;
  const cudaError_t e = device_status_ptr(&status);
  if (e != cudaSuccess) return e;
  const Keep k{a.c, a.table, a.kv_lens, a.cu_q, a.path, a.table_stride, a.total_q, a.max_q, status};
  const dim3 grid(a.batch, 2 * a.c.heads);
  return a.dim == 64 ? launch(keep_kernel<64>, grid, KT, 0, s, k) : launch(keep_kernel<128>, grid, KT, 0, s, k);
}

}  // namespace kv8
}  // namespace w4
