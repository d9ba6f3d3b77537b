// Attention over the 8-bit cache for many rows: prompts and prompt chunks.
//
// Bound by the two products. A CTA takes 256 rows of one sequence and kv head
// (row r: token r / group, head r % group, so grouped heads fill a tile too) as
// two tiles of 128, and walks the keys in steps of 128 tokens:
//   S = Q K^T   tcgen05.mma kind::f16, both operands in shared memory
//   P = 2^(S f + log2(vs) - m) in fp16, written over S in tensor memory
//   O += P V    A operand from tensor memory, V as stored (MN-major)
// with the two tiles half a step apart, so that one tile's products run under
// the other's exponentials. TMEM: S / P of the tiles 0-255, O 256-511.
//
// Roles (512 threads): warps 0-7 a row a thread: they scale Q to fp16, and turn S
// into P; warps 8-11 bring in the pages and widen the e4m3 codes to fp16
// (exactly) into the swizzled operand tiles, one layout for K (K-major) and V
// (MN-major); warp 12 issues the products. Registers go where they are needed
// (setmaxnreg 184 / 184 / 104 / 40: four times the 128 of the launch).
//
// The base m of a row's exponents is raised only when a score passes it by more
// than 8: then its warp rescales its rows of O in tensor memory, which has to
// wait for the tile's last product; otherwise it never touches O.
//
// Every mbarrier wait is bounded (one second): a timed-out wait records
// W4_ERR_TIMEOUT in the device status word and raises the CTA's abort flag; every
// role then leaves its loop, the issuer lets its products finish, and the tensor
// memory is freed.
#include <algorithm>
#include <mutex>

#include "decode_common.cuh"
#include "kv8_attention.cuh"

namespace w4 {
namespace kv8 {
namespace {

using namespace sm100;
using dec::bounded_wait;
using dec::drain_wait;

constexpr int TILE_ROWS = 128, CTA_ROWS = 256, KT = 128, THREADS = 512, KV_STAGES = 2;
constexpr int SOFT = 256, CONV = 128;  // threads of the roles
constexpr int TMEM_COLS = 512;
constexpr int BLK = 128 * 128;         // a block of 128 rows of 128 bytes (64 fp16 columns)
constexpr int SB = KT / 16;            // sixteens of a step: each lies in one page
constexpr int SLOTS = 4;               // steps whose scales are kept: a step's rows are done with
                                       // them when the keys three steps on are brought in

struct Prompt {
  Attn a;
  int tiles;  // of the longest sequence, of CTA_ROWS rows
};

template <int D>
struct PLayout {
  static constexpr int NB = D / 64;                        // 64-column blocks
  static constexpr int OFF_K = 2 * NB * BLK;               // after Q of both tiles
  static constexpr int OFF_V = OFF_K + KV_STAGES * NB * BLK;
  static constexpr int OFF_SC = OFF_V + KV_STAGES * NB * BLK;  // [slot][SB] {ks, log2 vs, 1/vs, 0}
  static constexpr int OFF_NAN = OFF_SC + SLOTS * SB * 16;      // [slot][4] tokens with a NaN value
  static constexpr int OFF_BAR = OFF_NAN + SLOTS * 16;
  static constexpr int BARS = 4 * KV_STAGES + 8;
  static constexpr int OFF_MISC = OFF_BAR + 8 * BARS;
  static constexpr int BYTES = OFF_MISC + 16 + 1024;       // + slack to align the base
};

struct PBars {
  uint32_t base;
  __device__ uint32_t kfull(int s) const { return base + 8 * s; }
  __device__ uint32_t kfree(int s) const { return base + 8 * (KV_STAGES + s); }
  __device__ uint32_t vfull(int s) const { return base + 8 * (2 * KV_STAGES + s); }
  __device__ uint32_t vfree(int s) const { return base + 8 * (3 * KV_STAGES + s); }
  __device__ uint32_t sfull(int i) const { return base + 8 * (4 * KV_STAGES + i); }      // S of tile i
  __device__ uint32_t pfull(int i) const { return base + 8 * (4 * KV_STAGES + 2 + i); }  // P of tile i
  __device__ uint32_t odone(int i) const { return base + 8 * (4 * KV_STAGES + 4 + i); }  // P V of tile i
  __device__ uint32_t qfull() const { return base + 8 * (4 * KV_STAGES + 6); }
  __device__ uint32_t drained() const { return base + 8 * (4 * KV_STAGES + 7); }  // only after a timeout
};

// Byte of 16-byte chunk c (of 8) of row r in a swizzled block.
__device__ __forceinline__ uint32_t sw(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }

// V as the B operand, MN-major: rows of tokens, 64 head columns (128 bytes) a
// row, 8-row groups of 1024 bytes (the stride along K), 64-column blocks BLK
// apart (the stride along N).
__device__ __forceinline__ uint64_t desc_v(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFF);
  d |= (uint64_t)(BLK >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
// D[tmem] (+)= A[tmem] * B[smem], fp16 operands.
__device__ __forceinline__ void umma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
      "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// A score's factor, kept above zero: a masked score of -inf times it stays -inf.
__device__ __forceinline__ float factor(float fr, float ks) { return fmaxf(fr * ks, 1.17549435e-38f); }

template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

template <int D, bool BF16>
__global__ void __launch_bounds__(THREADS, 1) prompt_kernel(const __grid_constant__ Prompt p) {
  using L = PLayout<D>;
  constexpr int NB = L::NB;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_addr(smem);
  const Attn& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const PBars bars{sbase + L::OFF_BAR};
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_MISC + 4);

  grid_wait();
  grid_launch_dependents();
  // the longest rows first: a causal sequence's last tile sees the most
  const int items = a.batch * a.c.heads;
  const int tile = p.tiles - 1 - blockIdx.x / items, bh = blockIdx.x % items;
  const int b = bh / a.c.heads, h = bh - b * a.c.heads;
  const Seq s = load_seq(a, b);
  if (!s.ok && tid == 0 && tile == 0) record(a.status, W4_ERR_PAGE);
  const int rows = s.n * a.group, row0 = tile * CTA_ROWS;
  if (row0 >= rows) return;

  if (tid == 0) {
    for (int i = 0; i < KV_STAGES; ++i) {
      mbar_init(bars.kfull(i), CONV);
      mbar_init(bars.vfull(i), CONV);
      mbar_init(bars.kfree(i), 1);
      mbar_init(bars.vfree(i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bars.sfull(i), 1);
      mbar_init(bars.pfull(i), SOFT / 2);
      mbar_init(bars.odone(i), 1);
    }
    mbar_init(bars.qfull(), SOFT);
    mbar_init(bars.drained(), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 12) {
    tmem_alloc(smem_addr(tmem_holder), TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;

  // tokens that a tile's last row sees, and its steps (tile 1 has the later rows)
  auto tokens_of = [&](int i) {
    const int first = row0 + TILE_ROWS * i;
    if (first >= rows) return 0;
    const int tok = (min(rows, first + TILE_ROWS) - 1) / a.group;
    return a.causal ? max(0, min(s.kv, s.kv - s.n + tok + 1)) : s.kv;
  };
  const int steps0 = (tokens_of(0) + KT - 1) / KT, steps1 = (tokens_of(1) + KT - 1) / KT;
  const int steps = max(steps0, steps1);
  // tokens from which on some row of the CTA does not see all
  const int first_lim = a.causal ? max(0, min(s.kv, s.kv - s.n + row0 / a.group + 1)) : s.kv;

  if (warp < 8) {
    // ------------------------------------------------------------ rows: Q, then S to P
    more_registers<184>();
    const int i = warp >> 2, quarter = warp & 3;
    const int lrow = quarter * 32 + lane, row = row0 + TILE_ROWS * i + lrow;
    const bool real = row < rows;
    const int tok = real ? row / a.group : 0;
    const int lim = !real ? 0 : a.causal ? min(s.kv, s.kv - s.n + tok + 1) : s.kv;
    const int my_steps = i ? steps1 : steps0;
    float fr;
    {
      const uint16_t* src = a.q + (size_t)(s.q0 + tok) * a.q_stride +
                            (size_t)(h * a.group + (real ? row - tok * a.group : 0)) * D;
      uint4 x[D / 8];
      float amax = 0.f;
#pragma unroll
      for (int c = 0; c < D / 8; ++c) x[c] = *reinterpret_cast<const uint4*>(src + 8 * c);
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        const uint32_t w[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
          amax = fmaxf(amax, fmaxf(fabsf(to_float<BF16>((uint16_t)(w[k] & 0xFFFF))),
                                   fabsf(to_float<BF16>((uint16_t)(w[k] >> 16)))));
      }
      // fp16 scaled to [2^14, 2^15); a negative scale goes into Q, so that fr >= 0
      const int e = max((int)(__float_as_uint(amax) >> 23) - 127, -100);
      const float up = copysignf(e < 128 ? pow2f(14 - e) : 1.f, a.scale_log2);
      fr = fabsf(a.scale_log2) * (e < 128 ? pow2f(e - 14) : 1.f);
      uint8_t* q = smem + i * NB * BLK;
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        const uint32_t w[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
        uint32_t y[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          y[k] = pack_f16(to_float<BF16>((uint16_t)(w[k] & 0xFFFF)) * up,
                          to_float<BF16>((uint16_t)(w[k] >> 16)) * up);
        *reinterpret_cast<uint4*>(q + (c / 8) * BLK + sw(lrow, c % 8)) = make_uint4(y[0], y[1], y[2], y[3]);
      }
      fence_proxy_async_smem();
      mbar_arrive(bars.qfull());
    }
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const uint32_t st = tmem + lanes + 128 * i, ot = tmem + lanes + 256 + D * i;
    float m = 0.f, room = NEG_INF, l = 0.f;
    bool ok = true;
    for (int j = 0; j < my_steps; ++j) {
      const int stage = j % KV_STAGES;
      ok = bounded_wait(bars.kfull(stage), (j / KV_STAGES) & 1, abort_flag, a.status) &&
           bounded_wait(bars.sfull(i), j & 1, abort_flag, a.status);
      ok = __all_sync(~0u, ok);
      if (!ok) break;
      tc_fence_after();
      uint32_t x[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(st + 32 * c, x[c]);
      const float4* sc = reinterpret_cast<const float4*>(smem + L::OFF_SC) + (j % SLOTS) * SB;
      tmem_ld_wait();
      if (KT * j + KT > first_lim) {  // some row does not see every token
        const uint32_t* nan = reinterpret_cast<const uint32_t*>(smem + L::OFF_NAN) + (j % SLOTS) * 4;
        const int left = lim - KT * j;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t bad = nan[c];
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            if (bad >> k & 1) x[c][k] = 0x7FFFFFFFu;
            if (32 * c + k >= left) x[c][k] = __float_as_uint(NEG_INF);
          }
        }
      }
      // the row's largest exponent, relative to m
      float top = NEG_INF;
#pragma unroll
      for (int g = 0; g < SB; ++g) {
        float y = NEG_INF;
#pragma unroll
        for (int k = 0; k < 16; ++k) y = fmaxf(y, __uint_as_float(x[g / 2][16 * (g & 1) + k]));
        const float4 z = sc[g];
        top = fmaxf(top, y * factor(fr, z.x) + z.y);
      }
      top -= m;
      if (__any_sync(~0u, top > room)) {
        const bool first = room == NEG_INF;
        float up = 0.f;
        if (top != NEG_INF && (first || top > 0.f)) {
          up = top;
          room = 8.f;
        }
        m += up;
        const float f = first ? 0.f : ex2(-up);
        l *= f;
        if (j > 0) {
          ok = __all_sync(~0u, bounded_wait(bars.odone(i), (j - 1) & 1, abort_flag, a.status));
          if (!ok) break;
          tc_fence_after();
          // (before a row's first score O holds zeros, which f = 0 keeps)
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t y[32];
            tmem_ld32(ot + 32 * c, y);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 32; ++k) y[k] = __float_as_uint(__uint_as_float(y[k]) * f);
            tmem_st32(ot + 32 * c, y);
          }
          tmem_st_wait();
        }
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t y[32];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int g = 4 * c + q;
          const float4 z = sc[g];
          const float f = factor(fr, z.x), add = z.y - m;
          float sum = 0.f;
#pragma unroll
          for (int k = 0; k < 16; k += 2) {
            const float s0 = __uint_as_float(x[g / 2][16 * (g & 1) + k]);
            const float s1 = __uint_as_float(x[g / 2][16 * (g & 1) + k + 1]);
            float p0 = ex2(s0 * f + add), p1 = ex2(s1 * f + add);
            sum += p0 + p1;
            y[8 * q + k / 2] = pack_f16(p0, p1);
          }
          l += sum * z.z;
        }
        tmem_st32(st + 32 * c, y);
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(bars.pfull(i));
    }
    if (ok && my_steps > 0)
      ok = __all_sync(~0u, bounded_wait(bars.odone(i), (my_steps - 1) & 1, abort_flag, a.status));
    if (ok) {
      tc_fence_after();
      const float inv = l == 0.f ? 0.f : 1.f / l;
      uint16_t* dst = a.out + ((size_t)(s.q0 + tok) * a.q_heads + h * a.group + (row - tok * a.group)) * D;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t y[32];
        if (my_steps > 0) {
          tmem_ld32(ot + 32 * c, y);
          tmem_ld_wait();
        }
        if (!real) continue;
#pragma unroll
        for (int k = 0; k < 32; k += 8) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            w[e] = my_steps > 0 ? pack_out<BF16>(__uint_as_float(y[k + 2 * e]) * inv,
                                                 __uint_as_float(y[k + 2 * e + 1]) * inv)
                                : 0u;
          *reinterpret_cast<uint4*>(dst + 32 * c + k) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
  } else if (warp < 12) {
    // ------------------------------------------------------------ pages to operand tiles
    fewer_registers<104>();
    const int c = tid - SOFT, p4 = c & 3, r32 = c >> 2;  // 16-byte piece p4 (+ 4 n), row r32 (+ 32 i)
    const int shift = a.c.page_shift, mask = (1 << shift) - 1;
    const int32_t* table = a.table + (size_t)b * a.table_stride;
    float4* sc = reinterpret_cast<float4*>(smem + L::OFF_SC);
    uint8_t* nan = smem + L::OFF_NAN;
    // row of the cache that holds token j (-1: none)
    auto cache_row = [&](int j) {
      if (j >= s.kv) return -1;
      const int pg = table[j >> shift];
      if ((unsigned)pg >= (unsigned)a.c.pages) {
        record(a.status, W4_ERR_PAGE);
        return -1;
      }
      return ((pg * a.c.heads + h) << shift) + (j & mask);  // below 2^31
    };
    uint4 kr[4][NB], vr[4][NB];
    auto load = [&](uint4 (&raw)[4][NB], const uint8_t* base, const int (&at)[4]) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int n = 0; n < NB; ++n)
          raw[i][n] = at[i] >= 0 ? dec::ldg_x(reinterpret_cast<const uint16_t*>(base + (size_t)at[i] * D + 64 * n + 16 * p4))
                                 : make_uint4(0, 0, 0, 0);
    };
    auto widen = [&](const uint4 (&raw)[4][NB], uint8_t* to) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          const uint32_t w[4] = {raw[i][n].x, raw[i][n].y, raw[i][n].z, raw[i][n].w};
          uint32_t y[8];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            y[2 * k] = e4m3x2_to_f16x2((uint16_t)(w[k] & 0xFFFF));
            y[2 * k + 1] = e4m3x2_to_f16x2((uint16_t)(w[k] >> 16));
          }
          const int r = 32 * i + r32;
          *reinterpret_cast<uint4*>(to + n * BLK + sw(r, 2 * p4)) = make_uint4(y[0], y[1], y[2], y[3]);
          *reinterpret_cast<uint4*>(to + n * BLK + sw(r, 2 * p4 + 1)) = make_uint4(y[4], y[5], y[6], y[7]);
        }
    };
    // Codes are loaded a step ahead of their use, table entries two, scales (threads
    // 0-7: a sixteen each) like the codes.
    int at[4], sat = -1;
    float ks = 0.f, vs = 1.f;
    auto rows_at = [&](int j) {
#pragma unroll
      for (int i = 0; i < 4; ++i) at[i] = j < steps ? cache_row(KT * j + 32 * i + r32) : -1;
      if (c < SB) sat = j < steps ? cache_row(KT * j + 16 * c) : -1;
    };
    auto load_scales = [&]() {
      ks = sat < 0 ? 0.f : a.c.ks[sat >> shift];
      vs = sat < 0 ? 1.f : a.c.vs[sat >> shift];
    };
    rows_at(0);
    load(kr, a.c.k, at);
    load(vr, a.c.v, at);
    bool none = sat < 0;
    load_scales();
    rows_at(1);
    for (int j = 0; j < steps; ++j) {
      const int stage = j % KV_STAGES, slot = j % SLOTS;
      const uint32_t ph = ((j / KV_STAGES) & 1) ^ 1;
      if (!__all_sync(~0u, bounded_wait(bars.kfree(stage), ph, abort_flag, a.status))) break;
      if (c < SB) {
        sc[slot * SB + c] = make_float4(ks, none ? NEG_INF : __log2f(vs), __fdividef(1.f, vs), 0.f);
        none = sat < 0;
        load_scales();
      }
      widen(kr, smem + L::OFF_K + stage * NB * BLK);
      fence_proxy_async_smem();
      load(kr, a.c.k, at);
      if (KT * j + KT > first_lim) {
        // Some row does not see every token, and 0 * NaN is NaN: NaN values leave the
        // operand and come back through the scores of the rows that see them.
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          bool hit = false;
#pragma unroll
          for (int n = 0; n < NB; ++n) {
            hit |= zero_nan_codes(vr[i][n].x);
            hit |= zero_nan_codes(vr[i][n].y);
            hit |= zero_nan_codes(vr[i][n].z);
            hit |= zero_nan_codes(vr[i][n].w);
          }
          // a warp has eight tokens, four lanes each: one byte of the 32 tokens' word
          uint32_t bits = __ballot_sync(~0u, hit);
          bits |= bits >> 1;
          bits |= bits >> 2;
          bits &= 0x11111111u;
          uint32_t byte = 0;
#pragma unroll
          for (int k = 0; k < 8; ++k) byte |= (bits >> (4 * k) & 1) << k;
          if (lane == 0) nan[slot * 16 + 4 * i + (warp - 8)] = (uint8_t)byte;
        }
      }
      mbar_arrive(bars.kfull(stage));
      if (!__all_sync(~0u, bounded_wait(bars.vfree(stage), ph, abort_flag, a.status))) break;
      widen(vr, smem + L::OFF_V + stage * NB * BLK);
      fence_proxy_async_smem();
      mbar_arrive(bars.vfull(stage));
      load(vr, a.c.v, at);
      rows_at(j + 2);
    }
  } else {
    // ------------------------------------------------------------ products
    fewer_registers<40>();
    if (warp == 12 && lane == 0) {
      constexpr uint32_t IDESC_S = idesc_f16(0, TILE_ROWS, KT);
      constexpr uint32_t IDESC_O = idesc_f16(0, TILE_ROWS, D) | (1u << 16);  // V is MN-major
      bool ok = bounded_wait(bars.qfull(), 0, abort_flag, a.status), issued = false;
      auto scores = [&](int i, int j) {  // S of tile i, step j
        const int stage = j % KV_STAGES;
        if (!(ok = ok && bounded_wait(bars.kfull(stage), (j / KV_STAGES) & 1, abort_flag, a.status))) return;
        tc_fence_after();
        const uint32_t qa = sbase + i * NB * BLK, ka = sbase + L::OFF_K + stage * NB * BLK;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = (k / 4) * BLK + (k % 4) * 32;
          umma_f16(tmem + 128 * i, smem_desc_k128(qa + off), smem_desc_k128(ka + off), IDESC_S, k != 0);
        }
        issued = true;
        umma_commit(bars.sfull(i));
        // the stage is free once the last tile that uses it has read it
        if (i == 1 || j >= steps1) umma_commit(bars.kfree(stage));
      };
      if (steps0 > 0) scores(0, 0);
      if (steps1 > 0) scores(1, 0);
      for (int j = 0; ok && j < steps; ++j) {
        const int stage = j % KV_STAGES;
        for (int i = 0; ok && i < 2; ++i) {
          const int n = i ? steps1 : steps0;
          if (j >= n) continue;
          if (!(ok = bounded_wait(bars.vfull(stage), (j / KV_STAGES) & 1, abort_flag, a.status) &&
                     bounded_wait(bars.pfull(i), j & 1, abort_flag, a.status)))
            break;
          tc_fence_after();
          const uint32_t va = sbase + L::OFF_V + stage * NB * BLK;
#pragma unroll
          for (int k = 0; k < KT / 16; ++k)
            umma_f16_ts(tmem + 256 + D * i, tmem + 128 * i + 8 * k, desc_v(va + k * 2048), IDESC_O,
                        j != 0 || k != 0);
          umma_commit(bars.odone(i));
          if (i == 1 || j >= steps1) umma_commit(bars.vfree(stage));
          if (j + 1 < n) scores(i, j + 1);
        }
      }
      if (!ok && issued) {  // let what was issued finish before the memory goes
        umma_commit(bars.drained());
        drain_wait(bars.drained(), 0);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

template <int D, bool BF16>
cudaError_t launch_it(const Prompt& p, cudaStream_t s) {
  static bool done[64] = {};
  constexpr int bytes = PLayout<D>::BYTES;
  cudaError_t e = allow_smem(prompt_kernel<D, BF16>, bytes, done);
  if (e != cudaSuccess) return e;
  const long long grid = (long long)p.tiles * p.a.c.heads * p.a.batch;
  if (grid >= (1ll << 31)) return cudaErrorInvalidValue;
  return launch(prompt_kernel<D, BF16>, dim3((unsigned)grid), THREADS, bytes, s, p);
}

}  // namespace

cudaError_t launch_prompt(const Attn& a, int dim, int bf16, cudaStream_t s) {
  Prompt p;
  p.a = a;
  p.tiles = (int)(((long long)a.max_q * a.group + CTA_ROWS - 1) / CTA_ROWS);
  if (dim == 64) return bf16 ? launch_it<64, true>(p, s) : launch_it<64, false>(p, s);
  return bf16 ? launch_it<128, true>(p, s) : launch_it<128, false>(p, s);
}

}  // namespace kv8
}  // namespace w4
