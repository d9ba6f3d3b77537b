// Attention over the 8-bit key-value cache.
//
//   out[i][h] = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q . k_j),
//   k_j = kc_j ks, v_j = vc_j vs  (ks, vs: one scale per page and head).
//
// One pass over the cache with a running maximum. With x_j = log2(e) scale ks
// (q . kc_j) + log2(vs) the running maximum is m = max x_j, p'_j = 2^(x_j - m),
// and
//   O = sum_j p'_j vc_j,   l = sum_j p'_j / vs,   out = O / l:
// the values' scale enters the exponent, so the codes themselves are the
// operand of the second product and p' <= 1 fits fp16.
//
// The q_heads / kv_heads query heads that share a kv head, and the new tokens
// of a sequence, are rows of one item: row r is token r / group, head r % group.
#include "kv8_device.cuh"

namespace w4 {
namespace kv8 {
namespace {

constexpr int WARPS = 4, THREADS = WARPS * 32, ROWS = 16, STEP = 32;
constexpr float NEG_INF = -__builtin_huge_valf();

struct Attn {
  const uint16_t* q;
  size_t q_stride;
  Cache c;
  const int32_t *table, *kv_lens, *cu_q;
  uint16_t* out;
  int table_stride, batch, total_q, max_q, max_kv, q_heads, group, causal;
  float scale_log2;  // scale * log2(e)
  int row_tiles;     // of the longest sequence
  int* status;
};

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

// Sequence b of the batch, checked: rows of new tokens and cached tokens.
struct Seq {
  int q0, n, kv;
  bool ok;
};
__device__ __forceinline__ Seq load_seq(const Attn& a, int b) {
  Seq s;
  s.q0 = a.cu_q[b];
  s.n = a.cu_q[b + 1] - s.q0;
  s.kv = a.kv_lens[b];
  s.ok = s.q0 >= 0 && s.n >= 0 && s.n <= a.max_q && s.q0 <= a.total_q - s.n;
  if (!s.ok) s.n = 0;
  if (s.kv < 0 || s.kv > a.max_kv || s.kv > ((long long)a.table_stride << a.c.page_shift)) {
    s.kv = 0;
    s.ok = false;
  }
  return s;
}

// One CTA: 16 rows of one sequence and kv head over all their tokens; the warps
// take steps of 32 tokens in turn, each with its own maximum and sums, merged at
// the end through shared memory.
template <int D, bool BF16>
__global__ void __launch_bounds__(THREADS) rows_kernel(const Attn a) {
  constexpr int KS = D / 16;   // k-steps of q . k
  constexpr int NT = D / 8;    // column tiles of p . v
  constexpr int CH = D / 64;   // 16-byte pieces of a key row a lane takes
  constexpr int OS = D + 4;    // row pitch of the merge buffer
  __shared__ float o_sh[WARPS][ROWS][OS];
  __shared__ float m_sh[WARPS][ROWS], l_sh[WARPS][ROWS];
  grid_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int tile = blockIdx.x % a.row_tiles, bh = blockIdx.x / a.row_tiles;
  const int b = bh / a.c.heads, h = bh - b * a.c.heads;
  const Seq s = load_seq(a, b);
  if (!s.ok && threadIdx.x == 0) record(a.status, W4_ERR_PAGE);
  const int rows = s.n * a.group;
  if (tile * ROWS >= rows) return;

  // this lane's rows g and g + 8: queries as fp16 scaled to [2^14, 2^15)
  uint32_t qf[KS][4];
  float fr[2];
  int lim[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = tile * ROWS + g + 8 * i;
    const bool real = r < rows;
    const int tok = real ? r / a.group : 0;
    lim[i] = !real ? 0 : a.causal ? min(s.kv, s.kv - s.n + tok + 1) : s.kv;
    const uint16_t* src = a.q + (size_t)(s.q0 + tok) * a.q_stride +
                          (size_t)(h * a.group + (real ? r - tok * a.group : 0)) * D;
    float f[CH][16];
    float amax = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const uint4 x = *reinterpret_cast<const uint4*>(src + 64 * c + 16 * t + 8 * v);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          f[c][8 * v + 2 * j] = to_float<BF16>((uint16_t)(w[j] & 0xFFFF));
          f[c][8 * v + 2 * j + 1] = to_float<BF16>((uint16_t)(w[j] >> 16));
        }
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) amax = fmaxf(amax, fabsf(f[c][j]));
    }
    amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 2));
    const int e = max((int)(__float_as_uint(amax) >> 23) - 127, -100);  // amax in [2^e, 2^(e+1))
    const float up = e < 128 ? pow2f(14 - e) : 1.f;
    fr[i] = a.scale_log2 * (e < 128 ? pow2f(e - 14) : 1.f);
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      const float* x = &f[k / 4][4 * (k % 4)];
      qf[k][i] = pack_f16(x[0] * up, x[1] * up);
      qf[k][2 + i] = pack_f16(x[2] * up, x[3] * up);
    }
  }
  // the tile's last row sees the most
  const int last_tok = (min(rows, tile * ROWS + ROWS) - 1) / a.group;
  const int end = a.causal ? min(s.kv, s.kv - s.n + last_tok + 1) : s.kv;
  const int first_lim = a.causal ? s.kv - s.n + tile * ROWS / a.group + 1 : s.kv;

  float o[NT][4];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
  float m[2] = {NEG_INF, NEG_INF}, l[2] = {0.f, 0.f};
  const int shift = a.c.page_shift;
  for (int j0 = warp * STEP; j0 < end; j0 += WARPS * STEP) {
    uint4 kq[4][CH];
    uint32_t vq[2][4][D / 32];
    float ksc[2], vsc[2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int j = j0 + 16 * half;
      int p = j < s.kv ? a.table[(size_t)b * a.table_stride + (j >> shift)] : -1;
      if (p >= a.c.pages || (p < 0 && j < s.kv)) {
        if (lane == 0) record(a.status, W4_ERR_PAGE);
        p = -1;
      }
      const size_t ph = p < 0 ? 0 : (size_t)p * a.c.heads + h;
      const int slot = j & ((1 << shift) - 1);
      const uint8_t* kp = a.c.k + ((ph << shift) + slot) * D;
      const uint8_t* vp = a.c.v + ((ph << shift) + slot) * D;
      ksc[half] = p < 0 ? NEG_INF : a.c.ks[ph];
      vsc[half] = p < 0 ? 1.f : a.c.vs[ph];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = 8 * i + g;
#pragma unroll
        for (int c = 0; c < CH; ++c)
          kq[2 * half + i][c] = p >= 0 && j + row < s.kv
                                    ? *reinterpret_cast<const uint4*>(kp + row * D + 64 * c + 16 * t)
                                    : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 8 * (i >> 1) + 2 * t + (i & 1);
        const bool in = p >= 0 && j + row < s.kv;
        if constexpr (D == 128) {
          const uint4 x = in ? *reinterpret_cast<const uint4*>(vp + row * D + 16 * g)
                             : make_uint4(0, 0, 0, 0);
          vq[half][i][0] = x.x, vq[half][i][1] = x.y, vq[half][i][2] = x.z, vq[half][i][3] = x.w;
        } else {
          const uint2 x = in ? *reinterpret_cast<const uint2*>(vp + row * D + 8 * g)
                             : make_uint2(0, 0);
          vq[half][i][0] = x.x, vq[half][i][1] = x.y;
        }
      }
    }
    // Rows that see different tokens share the value operand, and 0 * NaN is NaN:
    // in a step that some rows see only in part, NaN values leave the operand and
    // come back through the scores of the rows that do see them.
    uint32_t nan_tokens = 0;
    if (j0 + STEP > first_lim) {
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int w = 0; w < D / 32; ++w)
            if (zero_nan_codes(vq[half][i][w]))
              nan_tokens |= 1u << (16 * half + 8 * (i >> 1) + 2 * t + (i & 1));
      nan_tokens = __reduce_or_sync(~0u, nan_tokens);
    }
    float x[4][4];
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      x[n][0] = x[n][1] = x[n][2] = x[n][3] = 0.f;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const uint32_t w[4] = {kq[n][c].x, kq[n][c].y, kq[n][c].z, kq[n][c].w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_f16(x[n], qf[4 * c + k], e4m3x2_to_f16x2((uint16_t)(w[k] & 0xFFFF)),
                  e4m3x2_to_f16x2((uint16_t)(w[k] >> 16)));
      }
    }
    float top[2] = {m[0], m[1]};
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const int half = n >> 1;
      const float lv = __log2f(vsc[half]);
      const bool none = ksc[half] == NEG_INF;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int col = j0 + 8 * n + 2 * t + (i & 1);
        float y = x[n][i] * (fr[i >> 1] * ksc[half]) + lv;
        if (nan_tokens >> (col - j0) & 1) y = __int_as_float(0x7FFFFFFF);
        x[n][i] = col < lim[i >> 1] && !none ? y : NEG_INF;
        top[i >> 1] = fmaxf(top[i >> 1], x[n][i]);
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      top[i] = fmaxf(top[i], __shfl_xor_sync(~0u, top[i], 1));
      top[i] = fmaxf(top[i], __shfl_xor_sync(~0u, top[i], 2));
      const float base = top[i] == NEG_INF ? 0.f : top[i];
      const float f = ex2(m[i] - base);
      m[i] = top[i];
      top[i] = base;
      l[i] *= f;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        o[n][2 * i] *= f;
        o[n][2 * i + 1] *= f;
      }
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint32_t pf[4];
      float sum[2] = {0.f, 0.f};
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        float* y = x[2 * half + n];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          y[i] = ex2(y[i] - top[i >> 1]);
          sum[i >> 1] += y[i];
        }
        pf[2 * n] = pack_f16(y[0], y[1]);
        pf[2 * n + 1] = pack_f16(y[2], y[3]);
      }
      const float iv = __fdividef(1.f, vsc[half]);
      l[0] += sum[0] * iv;
      l[1] += sum[1] * iv;
#pragma unroll
      for (int w = 0; w < D / 32; ++w) {
        const uint32_t* c0 = &vq[half][0][w];
        constexpr int R = D / 32;
        const uint32_t a01 = prmt(c0[0], c0[R], 0x5140), a23 = prmt(c0[0], c0[R], 0x7362);
        const uint32_t b01 = prmt(c0[2 * R], c0[3 * R], 0x5140), b23 = prmt(c0[2 * R], c0[3 * R], 0x7362);
        mma_f16(o[4 * w], pf, e4m3x2_to_f16x2((uint16_t)(a01 & 0xFFFF)), e4m3x2_to_f16x2((uint16_t)(b01 & 0xFFFF)));
        mma_f16(o[4 * w + 1], pf, e4m3x2_to_f16x2((uint16_t)(a01 >> 16)), e4m3x2_to_f16x2((uint16_t)(b01 >> 16)));
        mma_f16(o[4 * w + 2], pf, e4m3x2_to_f16x2((uint16_t)(a23 & 0xFFFF)), e4m3x2_to_f16x2((uint16_t)(b23 & 0xFFFF)));
        mma_f16(o[4 * w + 3], pf, e4m3x2_to_f16x2((uint16_t)(a23 >> 16)), e4m3x2_to_f16x2((uint16_t)(b23 >> 16)));
      }
    }
  }
  // lane (g, t) holds, of rows g and g + 8, the columns D/8 (2t + e) + n
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    l[i] += __shfl_xor_sync(~0u, l[i], 1);
    l[i] += __shfl_xor_sync(~0u, l[i], 2);
    if (t == 0) {
      m_sh[warp][g + 8 * i] = m[i];
      l_sh[warp][g + 8 * i] = l[i];
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) o_sh[warp][g + 8 * i][NT * (2 * t + e) + n] = o[n][2 * i + e];
  }
  __syncthreads();
  const int row = threadIdx.x >> 3, c0 = (threadIdx.x & 7) * (D / 8);
  const int r = tile * ROWS + row;
  if (r >= rows) return;
  float top = NEG_INF, sum = 0.f, acc[D / 8];
#pragma unroll
  for (int w = 0; w < WARPS; ++w) top = fmaxf(top, m_sh[w][row]);
#pragma unroll
  for (int n = 0; n < D / 8; ++n) acc[n] = 0.f;
  if (top != NEG_INF) {
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const float f = ex2(m_sh[w][row] - top);
      sum += l_sh[w][row] * f;
#pragma unroll
      for (int n = 0; n < D / 8; ++n) acc[n] += o_sh[w][row][c0 + n] * f;
    }
    const float inv = 1.f / sum;
#pragma unroll
    for (int n = 0; n < D / 8; ++n) acc[n] *= inv;
  }
  const int tok = r / a.group;
  uint16_t* dst = a.out + ((size_t)(s.q0 + tok) * a.q_heads + h * a.group + (r - tok * a.group)) * D + c0;
#pragma unroll
  for (int n = 0; n < D / 8; n += 8)
    *reinterpret_cast<uint4*>(dst + n) =
        make_uint4(pack_out<BF16>(acc[n], acc[n + 1]), pack_out<BF16>(acc[n + 2], acc[n + 3]),
                   pack_out<BF16>(acc[n + 4], acc[n + 5]), pack_out<BF16>(acc[n + 6], acc[n + 7]));
}

}  // namespace

size_t attention_workspace_bytes(int batch, int max_q, int max_kv, int q_heads, int kv_heads,
                                 int dim) {
  (void)batch, (void)max_q, (void)max_kv, (void)q_heads, (void)kv_heads, (void)dim;
  return 0;
}

cudaError_t launch_attention(const AttnArgs& a, cudaStream_t s) {
  int* status = nullptr;
  const cudaError_t e = device_status_ptr(&status);
  if (e != cudaSuccess) return e;
  const int group = a.q_heads / a.c.heads;
  const long long tiles = ((long long)a.max_q * group + ROWS - 1) / ROWS;
  const long long grid = tiles * a.c.heads * a.batch;
  if (grid >= (1ll << 31)) return cudaErrorInvalidValue;
  const Attn p{a.q, a.q_stride, a.c, a.table, a.kv_lens, a.cu_q, a.out, a.table_stride, a.batch,
               a.total_q, a.max_q, a.max_kv, a.q_heads, group, a.causal,
               a.scale * 1.44269504088896340736f, (int)tiles, status};
  const dim3 gr((unsigned)grid);
  if (a.dim == 64)
    return a.bf16 ? launch(rows_kernel<64, true>, gr, THREADS, 0, s, p)
                  : launch(rows_kernel<64, false>, gr, THREADS, 0, s, p);
  return a.bf16 ? launch(rows_kernel<128, true>, gr, THREADS, 0, s, p)
                : launch(rows_kernel<128, false>, gr, THREADS, 0, s, p);
}

}  // namespace kv8
}  // namespace w4
