// Device code shared by the two attention kernels of the 8-bit cache.
//
//   out[i][h] = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q . k_j),
//   k_j = kc_j ks, v_j = vc_j vs  (ks, vs: one scale per page and head).
//
// One pass over the cache with a running maximum. With x_j = log2(e) scale ks
// (q . kc_j) + log2(vs) the running base is m, p'_j = 2^(x_j - m + P_UP), and
//   O = sum_j p'_j vc_j,   l = sum_j p'_j / vs,   out = O / l:
// the values' scale enters the exponent, so the codes themselves are the
// operand of the second product, and what p' is scaled by cancels.
//
// p' is rounded to fp16 for that product (l takes it as it is). The base is raised to
// the largest x_j only when that passes it by more than P_ROOM, so the largest p' lies
// between 2^P_UP and 2^(P_UP + P_ROOM) = 2^15: a token's p' keeps 11 bits down to
// 2^-22 of the largest, and no more than 2^-33 of the largest is lost of a smaller one.
// With p' from 1 to 2^8 instead it was 2^-25: 131072 tokens with 2^-26 each of one
// token's weight were lost whole, and so were pages whose values' scale stands 2^26
// below another's. Room costs nothing here and what it leaves below is precision, but
// raising the base means rescaling O: a prompt of 8000 tokens took 448 us with P_ROOM
// 4, 434 with 5, 427 with 6, 418 with 7, 414 with 8 (P_UP = 15 - P_ROOM, 10 for 4).
//
// The q_heads / kv_heads query heads that share a kv head, and the new tokens
// of a sequence, are rows of one item: row r is token r / group, head r % group.
#pragma once

#include "decode_common.cuh"
#include "kv8_device.cuh"

namespace w4 {
namespace kv8 {

constexpr float NEG_INF = -__builtin_huge_valf();
constexpr float P_UP = 8.f, P_ROOM = 7.f;

// dec::bounded_wait for barriers that hand over every microsecond or less: the
// timer (a read of some hundred cycles) and the abort flag are looked at only
// after many tries, so a waiter sees the phase end at once.
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                         int* status) {
  if (__builtin_expect(sm100::mbar_try_wait(bar, parity), 1)) return true;
  uint64_t t0 = 0;
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (sm100::mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    const uint64_t t = sm100::globaltimer_ns();
    if (t0 == 0) t0 = t;
    if (t - t0 > dec::WAIT_LIMIT_NS) {
      *abort_flag = 1;
      atomicExch(status, W4_ERR_TIMEOUT);
      return false;
    }
  }
}

struct Attn {
  const uint16_t* q;
  size_t q_stride;
  Cache c;
  const int32_t *table, *kv_lens, *cu_q;
  uint16_t* out;
  int table_stride, batch, total_q, max_q, max_kv, q_heads, group, causal;
  float scale_log2;  // scale * log2(e)
  int* status;
};

// A tensor map over one side's token rows, a box `rows` of them high.
bool encode_rows(CUtensorMap* map, const void* base, const Cache& c, int D, int rows);

// The kernel for many rows (kv8_prompt.cu).
cudaError_t launch_prompt(const Attn& a, int dim, int bf16, void* workspace, cudaStream_t s);
size_t prompt_workspace_bytes(int batch, int max_q, int max_kv, int group, int kv_heads, int dim);

template <bool BF16>
__device__ __forceinline__ float to_float(uint16_t h) {
  if constexpr (BF16) return __uint_as_float((uint32_t)h << 16);
  else return __half2float(__ushort_as_half(h));
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack_out(float lo, float hi) {
  uint32_t d;
  if constexpr (BF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) { return pack_out<false>(lo, hi); }
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Sets the NaN codes (0x7F, 0xFF) of four to zero; whether there were any.
__device__ __forceinline__ bool zero_nan_codes(uint32_t& w) {
  const uint32_t hit = ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
  if (hit == 0) return false;
  w &= ~((hit >> 7) * 0xFFu);
  return true;
}

// Sequence b of the batch, checked: rows of new tokens and cached tokens. One past a
// bound has no cached tokens, so that its rows become zeros; one past max_q has more
// rows than the grids are made for (zero_rows, or units dealt by the rows there are).
struct Seq {
  int q0, n, kv;
  bool ok;
};
__device__ __forceinline__ Seq load_seq(const Attn& a, int b) {
  Seq s;
  s.q0 = a.cu_q[b];
  s.n = a.cu_q[b + 1] - s.q0;
  s.kv = a.kv_lens[b];
  s.ok = s.q0 >= 0 && s.n >= 0 && s.q0 <= a.total_q - s.n;
  if (!s.ok) s.n = 0;
  if (s.n > a.max_q || s.kv < 0 || s.kv > a.max_kv ||
      s.kv > ((long long)a.table_stride << a.c.page_shift)) {
    s.kv = 0;
    s.ok = false;
  }
  return s;
}

// Zeros to all rows of a sequence in the query heads of kv head h: a block's share.
template <int D>
__device__ void zero_rows(const Attn& a, const Seq& s, int h, int part, int parts) {
  const int width = a.group * (D / 8);  // 16-byte pieces of a token
  const long long all = (long long)s.n * width;
  for (long long i = (long long)part * blockDim.x + threadIdx.x; i < all; i += (long long)parts * blockDim.x) {
    const long long tok = i / width;
    reinterpret_cast<uint4*>(a.out + ((size_t)(s.q0 + tok) * a.q_heads + (size_t)h * a.group) * D)[i - tok * width] =
        make_uint4(0, 0, 0, 0);
  }
}

}  // namespace kv8
}  // namespace w4
