// Norms of query and key heads and the rotation by position, in one pass.
//
//   y = x * (mean(x^2) + eps)^-1/2 * w          (each head of each token; w optional)
//   (a, b) -> (a c - b s, b c + a s)            for the pairs of y's first `rot` elements,
//   (c, s) = table[position][j], table[position][rot / 2 + j] for pair j: elements j and
//   j + rot / 2, or (interleaved) 2 j and 2 j + 1.
//
// A thread has two 16-byte pieces of a head, chosen so that it has both elements of its
// pairs: nothing but the sum of squares crosses lanes. Half-split, thread l of a head's
// D / 16 has pieces l and l + rot / 16 while l < rot / 16; interleaved, or past what is
// rotated, 2 l and 2 l + 1. Either way its cosines are 8 l to 8 l + 7 of a table row.
//
// Everything is fp32 from the loads to the one rounding at the end.
//
// Bound by memory: a prompt of 8000 tokens of 32 + 8 heads of 128 (168 MB) takes 30 us,
// 5.6 TB/s (one of 4000, which fits in L2, 12.9 us); one token
// 1.7 us in a graph, a launch's latency. A thread that goes on to its next heads while
// their elements are on their way (registers for two shares) was no faster: 34 to 44 us.
#include "kv8_device.cuh"
#include "w4a16_device.cuh"

namespace w4 {
namespace kv8 {
namespace {

constexpr int THREADS = 64;  // (blocks of 256 end in steps: 31.4 against 30.0 us on a prompt of 8000)

constexpr float TINY = 0x1p-100f, TINY_UP = 0x1p80f;

struct Side {
  const uint16_t* in;
  uint16_t* out;
  size_t in_stride, out_stride;
  const float* weight;  // or nullptr: no norm
  int heads, teams;     // teams of a token
};
struct Rope {
  Side side[2];  // queries, keys
  const float* table;  // or nullptr: no rotation
  const int32_t* positions;
  int rows, rot, tokens;
  float eps;
  int* status;
};

template <bool BF16>
__device__ __forceinline__ void widen(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = half_bits_to_float<BF16>((uint16_t)(w[i] & 0xFFFF));
    f[2 * i + 1] = half_bits_to_float<BF16>((uint16_t)(w[i] >> 16));
  }
}
template <bool BF16>
__device__ __forceinline__ uint4 narrow(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
    else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}

// HEADS: of one token and side that a team of D / 16 threads takes, `teams` apart, so
// that neighbouring teams have neighbouring heads.
template <int D, bool BF16, bool INTERLEAVED, int HEADS>
__global__ void __launch_bounds__(THREADS) rope_kernel(const __grid_constant__ Rope r) {
  constexpr int TEAM = D / 16;
  grid_wait();
  grid_launch_dependents();
  const int l = threadIdx.x % TEAM;
  const int per = r.side[0].teams + r.side[1].teams;
  // the block's first team, and this thread's from there (one long division a block)
  const long long team0 = (long long)blockIdx.x * (THREADS / TEAM);
  const int tok0 = (int)(team0 / per);
  int slot = (int)(team0 - (long long)tok0 * per) + threadIdx.x / TEAM;
  const int tok = tok0 + slot / per;
  slot -= (tok - tok0) * per;
  const int which = slot >= r.side[0].teams;
  const Side& s = r.side[which];
  if (which) slot -= r.side[0].teams;
  const bool here = tok < r.tokens;
  const int pos = here && r.positions ? r.positions[tok] : 0;
  const bool turns = r.table && l < r.rot / 16;
  const int first = !INTERLEAVED && turns ? l : 2 * l, second = !INTERLEAVED && turns ? l + r.rot / 16 : 2 * l + 1;
  uint4 x[HEADS][2];  // (of padding too: its position is still on its way; read for the last time)
#pragma unroll
  for (int i = 0; i < HEADS; ++i) {
    const int h = slot + i * s.teams;
    x[i][0] = x[i][1] = make_uint4(0, 0, 0, 0);
    if (here && h < s.heads) {
      const uint16_t* from = s.in + (size_t)tok * s.in_stride + (size_t)h * D;
      x[i][0] = __ldcs(reinterpret_cast<const uint4*>(from + 8 * first));
      x[i][1] = __ldcs(reinterpret_cast<const uint4*>(from + 8 * second));
    }
  }
  // (whole teams drop out, but their lanes stay for the shuffles)
  bool live = here && pos >= 0;
  if (live && r.table && pos >= r.rows) {
    live = false;
    if (l == 0) record(r.status, W4_ERR_POSITION);
  }
  float c[8], sn[8], w[2][8];
  if (live && turns) {
    const float* row = r.table + (size_t)pos * r.rot + 8 * l;
    load8(row, c);
    load8(row + r.rot / 2, sn);
  }
  if (here && s.weight) {
    load8(s.weight + 8 * first, w[0]);
    load8(s.weight + 8 * second, w[1]);
  }
#pragma unroll
  for (int i = 0; i < HEADS; ++i) {
    float a[8], b[8];
    widen<BF16>(x[i][0], a);
    widen<BF16>(x[i][1], b);
    if (r.side[0].weight || r.side[1].weight) {  // (all lanes of a warp, for the shuffles)
      float sum = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) sum += a[k] * a[k] + b[k] * b[k];
#pragma unroll
      for (int d = TEAM / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
      float mean = sum * (1.f / D) + r.eps;
      if constexpr (BF16) {
        // Squares of elements below 2^-75 leave fp32, which tells where eps is as small (0,
        // say) and nothing larger stands beside them: such a head is taken 2^80 times.
        const bool tiny = s.weight && mean < TINY;
        if (r.eps < TINY && __any_sync(~0u, tiny)) {
          const float up = tiny ? TINY_UP : 1.f;
          sum = 0.f;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            a[k] *= up, b[k] *= up;
            sum += a[k] * a[k] + b[k] * b[k];
          }
#pragma unroll
          for (int d = TEAM / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
          if (tiny) mean = sum * (1.f / D) + r.eps * up * up;
        }
      }
      if (s.weight) {
        const float inv = rsqrtf(mean);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          a[k] *= inv * w[0][k];
          b[k] *= inv * w[1][k];
        }
      }
    }
    if (turns) {
      if constexpr (INTERLEAVED) {
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
          const float a0 = a[k], b0 = b[k];
          a[k] = a0 * c[k / 2] - a[k + 1] * sn[k / 2];
          a[k + 1] = a[k + 1] * c[k / 2] + a0 * sn[k / 2];
          b[k] = b0 * c[4 + k / 2] - b[k + 1] * sn[4 + k / 2];
          b[k + 1] = b[k + 1] * c[4 + k / 2] + b0 * sn[4 + k / 2];
        }
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float a0 = a[k];
          a[k] = a0 * c[k] - b[k] * sn[k];
          b[k] = b[k] * c[k] + a0 * sn[k];
        }
      }
    }
    const int h = slot + i * s.teams;
    if (live && h < s.heads) {
      uint16_t* to = s.out + (size_t)tok * s.out_stride + (size_t)h * D;
      *reinterpret_cast<uint4*>(to + 8 * first) = narrow<BF16>(a);
      *reinterpret_cast<uint4*>(to + 8 * second) = narrow<BF16>(b);
    }
  }
}

template <int D, bool BF16, bool INTERLEAVED, int HEADS>
cudaError_t launch_heads(Rope& r, cudaStream_t s) {
  constexpr int TEAMS = THREADS / (D / 16);  // of a block
  for (Side& side : r.side) side.teams = (side.heads + HEADS - 1) / HEADS;
  const long long teams = (long long)r.tokens * (r.side[0].teams + r.side[1].teams);
  return launch(rope_kernel<D, BF16, INTERLEAVED, HEADS>, dim3((unsigned)((teams + TEAMS - 1) / TEAMS)), THREADS, 0, s, r);
}

// How many heads a team takes: one while that leaves the GPU half empty, where latency
// counts; more where the table and the weights, 128 bytes a thread from the L1 cache for
// 64 of a head's, would be what the kernel waits for. In us, replayed in a graph, 40 heads
// of 128 (1 / 4 / 8 heads a team): 64 tokens 1.9 / 2.5 / 3.4, 200 2.4 / 2.6 / 3.4, 350
// 3.3 / 2.9 / 3.6, 1500 8.2 / 6.1 / 6.3, 4000 21.2 / 12.9 / 13.4, 5500 29.7 / 22.7 / 21.2,
// 8000 42.3 / 33.2 / 30.0; 32 heads of 64: 333 2.1 / 2.6 / 3.3, 1000 3.1 / 3.0 / 4.0, 8000
// 16.6 / 10.2 / 12.1, 16000 34.1 / 23.9 / 24.4.
constexpr long long FEW_THREADS = 100000, MANY_THREADS = 1400000;  // with one head a team

template <int D, bool BF16, bool INTERLEAVED>
cudaError_t launch_pick(Rope& r, cudaStream_t s) {
  const long long threads = (long long)r.tokens * (r.side[0].heads + r.side[1].heads) * (D / 16);
  if (threads <= FEW_THREADS) return launch_heads<D, BF16, INTERLEAVED, 1>(r, s);
  if (threads <= MANY_THREADS) return launch_heads<D, BF16, INTERLEAVED, 4>(r, s);
  return launch_heads<D, BF16, INTERLEAVED, 8>(r, s);
}

template <int D>
cudaError_t launch_d(Rope& r, int bf16, int interleaved, cudaStream_t s) {
  if (interleaved) return bf16 ? launch_pick<D, true, true>(r, s) : launch_pick<D, false, true>(r, s);
  return bf16 ? launch_pick<D, true, false>(r, s) : launch_pick<D, false, false>(r, s);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s) {
  Rope r;
  const cudaError_t e = device_status_ptr(&r.status);
  if (e != cudaSuccess) return e;
  for (int i = 0; i < 2; ++i)
    r.side[i] = {a.rows[i].in, a.rows[i].out, a.rows[i].in_stride, a.rows[i].out_stride, a.rows[i].weight, a.rows[i].heads, 0};
  r.table = a.table;
  r.positions = a.positions;
  r.rows = a.table_rows;
  r.rot = a.rot;
  r.tokens = a.tokens;
  r.eps = a.eps;
  return a.dim == 64 ? launch_d<64>(r, a.bf16, a.interleaved, s) : launch_d<128>(r, a.bf16, a.interleaved, s);
}

}  // namespace kv8
}  // namespace w4
