// Attention over the 8-bit cache for few rows: decode steps and drafted tokens.
//
// Bound by reading the cache once. 8 or 16 rows (the query heads of a kv head
// times the new tokens) are one item; its tokens are cut into units of 32. All
// units of the batch, in order of sequence, head and row tile, are dealt to the
// warps of the GPU in contiguous runs of equal cost, whatever the lengths are
// (an item costs its units and ITEM_COST more): a warp that covers an item whole
// writes its output, the parts of the others go to the workspace and a second
// kernel joins them (in the order of the tokens, so the result does not depend
// on timing). Joining in the first kernel, by whoever finishes an item's last
// part, measured 14 to 20 us a call, all of it on the critical path: the write,
// the fence, the count and the reads wait for one another. Where no sequence is
// longer than 512 tokens every item gets a CTA of its own, whose warps take units
// in turn and are joined in shared memory, and that is all.
//
// Each warp brings its units in by TMA through a ring of its own (keys and
// values, 128-byte swizzle, so that the 16-byte shared loads below are free of
// bank conflicts), with the table entry of the unit after next and the queries
// of the next item on their way meanwhile. Both products are computed
// transposed, S^T = K Q^T and O^T = V^T P^T, with the codes, widened to fp16 in
// registers (exactly), as the 16-row A operand of mma.sync m16n8k16 and the
// query rows as its 8 columns: a kv head rarely has more than 8 query heads,
// and rows that do not exist would otherwise cost half of every product. (Eight
// rows cannot fill a tcgen05 tile, and the kernel is bound by HBM.) P^T goes
// from the accumulator's layout to the operand's by 8 x 8 transposes.
//   Row c of an A operand's eight is token rho(c): rho spreads the rows that a
//   phase of eight lanes reads over all banks of the swizzled tile.
#include <algorithm>

#include "decode_common.cuh"
#include "kv8_attention.cuh"

namespace w4 {
namespace kv8 {
namespace {

using namespace sm100;
using dec::drain_wait;

constexpr int WARPS = 4, THREADS = WARPS * 32, STEP = 32, STAGES = 2;
constexpr int MAX_SMS = 160;       // that a split call uses
constexpr int MAX_SCAN = 2048;     // sequences of a split call: every CTA scans their lengths
// Sequences up to this long are not split. Not split against split, in us: 1 sequence
// of 32 heads on 32, 3.8 / 10.3 at 128 tokens, 6.6 / 11.2 at 512, 10.1 / 11.5 at 1024,
// 17.1 / 12.5 at 2048; 64 of 64 on 8, 8.1 / 13.7, 14.7 / 19.1, 28.0 / 33.6 and 47.5 /
// 54.2; 256 of 32 on 8, 26 / 19, 57 / 53, 92 / 95 and 165 / 179. Those are batches of
// one length, the best that can happen to a call that is not split: where lengths
// differ, its longest item is its time.
constexpr int ITEM_TOKENS = 512;
// Of a warp's run in a split call. 24 sequences of 35 to 3001 tokens, 1 to 6 new,
// groups of 7: 17.1 us with 3 and 4, 18.2 with 6, 21.6 with 10, 26.2 with 16.
constexpr int MIN_COST = 4;
// Two CTAs an SM keep 128 KB of copies in flight. Three (168 registers) measured
// slower: 51.3 against 42.1 us on 64 ragged sequences of up to 4096 tokens, 102.5
// against 95.9 us on two of 131072, whose warps then end further apart.
constexpr int CTAS_PER_SM = 2;
constexpr int MAX_WORKERS = MAX_SMS * CTAS_PER_SM * WARPS;
constexpr int ITEM_COST = 2;       // of an item beyond its units: queries, output, joining

struct Rows {
  CUtensorMap tk, tv;  // token rows [pages * heads * page][D] bytes, box min(page, 32) rows
  Attn a;
  float* part;  // [warp][2]: sums [rows][D], then maximum and l [rows][2]
  int* rec;     // [warp][8]: the item begun but not finished there (Begun)
  int row_tiles, split, bf16;
};

__host__ __device__ constexpr int part_floats(int D, int NB) { return 8 * NB * (D + 2); }

// An item that a warp begins and others go on with.
struct alignas(32) Begun {
  int slot;  // of the warp's two parts; -1: none
  int more;  // further warps
  int q0, rows, h, tile;
};

// A run of units [u0, u1) of one item.
struct Seg {
  int b, h, tile, tiles, units, u0, u1;
  Seq s;
  long long left;  // cost of the run from this item's part on
};

template <int ROWS>
__device__ __forceinline__ void count_items(const Attn& a, Seg& g) {
  g.tiles = (g.s.n * a.group + ROWS - 1) / ROWS;
  g.units = max(1, (g.s.kv + STEP - 1) / STEP);
}
template <int ROWS>
__device__ __forceinline__ void load_items(const Attn& a, Seg& g) {
  g.s = load_seq(a, g.b);
  count_items<ROWS>(a, g);
}

// The item's part of a run that begins `skip` into its cost.
__device__ __forceinline__ void cut(Seg& g, long long skip) {
  g.u0 = (int)max(0ll, skip - ITEM_COST);
  g.u1 = (int)min((long long)g.units, max(0ll, skip + g.left - ITEM_COST));
  g.left -= ITEM_COST + g.units - skip;
}

// The next part with a unit in it; false at the run's end.
template <int ROWS>
__device__ __forceinline__ bool next_seg(const Attn& a, Seg& g) {
  if (g.left <= ITEM_COST) return false;
  if (++g.tile >= g.tiles) {
    g.tile = 0;
    if (++g.h >= a.c.heads) {
      g.h = 0;
      do {
        if (++g.b >= a.batch) return false;
        load_items<ROWS>(a, g);
      } while (g.tiles == 0);
    }
  }
  cut(g, 0);
  return true;
}

__device__ __forceinline__ int rho(int c) { return ((c >> 1) | ((c >> 1 & 1) << 2)) ^ ((c & 1) << 2); }

// Bytes from a tile's base to 16-byte piece p of row r (TMA's swizzle).
template <int D>
__device__ __forceinline__ uint32_t piece(int r, int p) {
  if constexpr (D == 128) return r * 128 + ((p ^ (r & 7)) << 4);
  else return r * 64 + ((p ^ (r >> 1 & 3)) << 4);
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}
// An 8 x 8 matrix of 16-bit values, lane (g, t) holding elements (g, 2t) and
// (g, 2t + 1), transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// Counts as one of the barrier's arrivals once this thread's copies have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

template <int D, int NB>
struct Layout {
  static constexpr int TILE = STEP * D, STAGE = 2 * TILE, RING = STAGES * STAGE, ROWS = 8 * NB;
  static constexpr int OS = D + 2;  // row pitch of the merge buffer (floats)
  static constexpr int OFF_ML = WARPS * RING;
  static constexpr int OFF_SC = OFF_ML + 2 * WARPS * ROWS * 4;
  static_assert(WARPS * ROWS * OS * 4 <= WARPS * RING, "the merge buffer takes the place of the rings");
  static constexpr int OFF_BAR = OFF_SC + WARPS * STAGES * 16;
  static constexpr int OFF_MISC = OFF_BAR + WARPS * STAGES * 8;
  static constexpr int BYTES = OFF_MISC + 8 + WARPS * 32 + 1024;  // + slack to align the base
};

// The queries of an item, one row a lane (its operand's column): row 8 nb + g.
template <int D, int NB>
struct Queries {
  uint4 x[NB][D / 64][2];
  __device__ __forceinline__ void load(const Attn& a, const Seg& seg, int g, int t) {
    const int rows = seg.s.n * a.group;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int row = seg.tile * 8 * NB + 8 * nb + g;
      const int tok = row < rows ? row / a.group : 0;
      const uint16_t* src = a.q + (size_t)(seg.s.q0 + tok) * a.q_stride +
                            (size_t)(seg.h * a.group + (row < rows ? row - tok * a.group : 0)) * D;
#pragma unroll
      for (int c = 0; c < D / 64; ++c)
#pragma unroll
        for (int v = 0; v < 2; ++v) x[nb][c][v] = *reinterpret_cast<const uint4*>(src + 64 * c + 16 * t + 8 * v);
    }
  }
};

// Where row rr of an item goes.
template <int D>
__device__ __forceinline__ uint16_t* out_row(const Attn& a, const Seg& g, int rr) {
  const int tok = rr / a.group;
  return a.out + ((size_t)(g.s.q0 + tok) * a.q_heads + g.h * a.group + (rr - tok * a.group)) * D;
}

// SPLIT: every warp has a run of its own; otherwise a CTA has an item.
template <int D, int NB, bool BF16, bool SPLIT>
__global__ void __launch_bounds__(THREADS, CTAS_PER_SM) rows_kernel(const __grid_constant__ Rows r) {
  using L = Layout<D, NB>;
  constexpr int ROWS = L::ROWS;
  constexpr int CH = D / 64;   // 16-byte pieces of a key row a lane takes
  constexpr int MT = D / 16;   // 16-row tiles of O^T; k-steps of K Q^T
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const Attn& a = r.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  float* o_sh = reinterpret_cast<float*>(smem);
  float* m_sh = reinterpret_cast<float*>(smem + L::OFF_ML);
  float* l_sh = m_sh + WARPS * ROWS;
  const uint32_t ring = smem_addr(smem) + warp * L::RING;
  float* sc_sh = reinterpret_cast<float*>(smem + L::OFF_SC) + warp * STAGES * 4;
  const uint32_t bars = smem_addr(smem + L::OFF_BAR) + warp * STAGES * 8;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_MISC);

  if (lane == 0) {
    // arrivals: TMA, and two scales for each page of a unit
    for (int i = 0; i < STAGES; ++i) mbar_init(bars + 8 * i, a.c.page_shift == 4 ? 5 : 3);
    fence_mbar_init();
  }
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    prefetch_tmap(&r.tk);
    prefetch_tmap(&r.tv);
  }
  grid_wait();
  grid_launch_dependents();

  // ---- this CTA's range of units
  Seg seg;
  long long per = 0;
  bool any = true;
  if constexpr (!SPLIT) {
    const int bh = blockIdx.x / r.row_tiles;
    seg.tile = blockIdx.x - bh * r.row_tiles;
    seg.b = bh / a.c.heads;
    seg.h = bh - seg.b * a.c.heads;
    load_items<ROWS>(a, seg);
    if (!seg.s.ok && threadIdx.x == 0) record(a.status, W4_ERR_PAGE);
    if (seg.s.n > a.max_q) {
      zero_rows<D>(a, seg.s, seg.h, seg.tile, r.row_tiles);
      return;
    }
    if (seg.tile >= seg.tiles) return;
    seg.left = ITEM_COST + seg.units;
    cut(seg, 0);
    __syncthreads();
  } else {
    // the batch's costs, summed over the CTA; whoever holds the sequence that a
    // warp's run begins in tells it
    long long* sums = reinterpret_cast<long long*>(smem + L::OFF_MISC + 8);  // [WARPS]
    long long* runs = sums + WARPS;                                          // [WARPS]: offset in b
    int* seqs = reinterpret_cast<int*>(runs + WARPS);                        // [WARPS][4]: b, Seq
    const int per_t = (a.batch + THREADS - 1) / THREADS;
    const int b0 = min(a.batch, (int)threadIdx.x * per_t), b1 = min(a.batch, b0 + per_t);
    long long sum = 0;
    for (seg.b = b0; seg.b < b1; ++seg.b) {
      load_items<ROWS>(a, seg);
      if (!seg.s.ok && blockIdx.x == 0) record(a.status, W4_ERR_PAGE);
      sum += (long long)seg.tiles * a.c.heads * (ITEM_COST + seg.units);
    }
    long long inc = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long u = __shfl_up_sync(~0u, inc, d);
      if (lane >= d) inc += u;
    }
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    long long before = inc - sum, total = 0;
    for (int w = 0; w < WARPS; ++w) {
      if (w < warp) before += sums[w];
      total += sums[w];
    }
    const long long workers = (long long)gridDim.x * WARPS;
    per = max((long long)MIN_COST, (total + workers - 1) / workers);
    for (int w = 0; w < WARPS; ++w) {
      const long long lo = ((long long)blockIdx.x * WARPS + w) * per;
      if (lo < before || lo >= before + sum) continue;
      long long at = before;
      if (per_t == 1) seg.b = b0;  // its lengths are still here
      for (int b = b0; b < b1; ++b) {
        if (per_t > 1) {
          seg.b = b;
          load_items<ROWS>(a, seg);
        }
        const long long n = (long long)seg.tiles * a.c.heads * (ITEM_COST + seg.units);
        if (lo < at + n) {
          runs[w] = lo - at;
          seqs[4 * w] = seg.b, seqs[4 * w + 1] = seg.s.q0, seqs[4 * w + 2] = seg.s.n, seqs[4 * w + 3] = seg.s.kv;
          break;
        }
        at += n;
      }
    }
    __syncthreads();
    const long long lo = ((long long)blockIdx.x * WARPS + warp) * per;
    if (lane == 0) r.rec[(blockIdx.x * WARPS + warp) * 8] = -1;
    any = lo < total;
    if (any) {
      seg.b = seqs[4 * warp];
      seg.s = {seqs[4 * warp + 1], seqs[4 * warp + 2], seqs[4 * warp + 3], true};
      count_items<ROWS>(a, seg);
      const int item = (int)(runs[warp] / (ITEM_COST + seg.units));
      seg.h = item / seg.tiles;
      seg.tile = item - seg.h * seg.tiles;
      seg.left = min(per, total - lo);
      cut(seg, runs[warp] - (long long)item * (ITEM_COST + seg.units));
      while (any && seg.u0 >= seg.u1) any = next_seg<ROWS>(a, seg);  // only its begin lies here
    }
  }
  constexpr int STRIDE = SPLIT ? 1 : WARPS;
  const int phase = SPLIT ? 0 : warp;

  // ---- the warp's units, brought in STAGES ahead. `p` is the unit to bring in
  // next; lanes 0 and 1 hold the table entries of its two halves, loaded when
  // the unit before it was issued.
  const int shift = a.c.page_shift;
  const bool halves = shift == 4;  // a unit spans two pages of 16
  Seg ps = seg;
  int pu = seg.u0 + phase, pit = 0, page_reg = -2;
  bool more = any, ok = true;
  auto settle = [&]() {  // move to the next segment with a unit for this warp; fetch its pages
    while (pu >= ps.u1) {
      if (!next_seg<ROWS>(a, ps)) {
        more = false;
        return;
      }
      pu = ps.u0 + phase;
    }
    if (lane < 2) {
      const int j = pu * STEP + 16 * lane;
      page_reg = j < ps.s.kv ? a.table[(size_t)ps.b * a.table_stride + (j >> shift)] : -2;
    }
  };
  auto issue = [&]() {
    if (!more || !ok) return;
    const int st = pit % STAGES;
    const uint32_t bar = bars + 8 * st, dst = ring + st * L::STAGE;
    int pg = page_reg;
    if (pg != -2 && (unsigned)pg >= (unsigned)a.c.pages) {
      record(a.status, W4_ERR_PAGE);
      pg = -1;
    }
    const int ph = pg < 0 ? -1 : pg * a.c.heads + ps.h;  // page and head (rows stay below 2^31)
    const int p0 = __shfl_sync(~0u, ph, 0), p1 = halves ? __shfl_sync(~0u, ph, 1) : -1;
    if (lane == 0) {
      constexpr uint32_t HALF = L::TILE / 2;
      const uint32_t box = halves ? HALF : L::TILE;
      mbar_arrive_expect_tx(bar, (p0 >= 0 ? 2 * box : 0) + (p1 >= 0 ? 2 * box : 0));
      if (p0 >= 0) {
        const int y = (p0 << shift) + ((pu * STEP) & ((1 << shift) - 1));
        tma_load_2d(dst, &r.tk, bar, 0, y);
        tma_load_2d(dst + L::TILE, &r.tv, bar, 0, y);
      }
      if (p1 >= 0) {
        tma_load_2d(dst + HALF, &r.tk, bar, 0, p1 << shift);
        tma_load_2d(dst + L::TILE + HALF, &r.tv, bar, 0, p1 << shift);
      }
    }
    if (lane < (halves ? 4 : 2)) {  // scales: keys and values of half 0, of half 1 (-inf: no page)
      const int p = lane < 2 ? p0 : p1;
      float* to = sc_sh + st * 4 + lane;
      if (p >= 0) {
        cp_async4(smem_addr(to), ((lane & 1) ? a.c.vs : a.c.ks) + p);
        cp_async_arrive(bar);
      } else {
        *to = (lane & 1) ? 1.f : NEG_INF;
        mbar_arrive(bar);
      }
    }
    ++pit;
    pu += STRIDE;
    settle();
  };
  if (any) settle();
#pragma unroll
  for (int i = 0; i < STAGES; ++i) issue();

  int it = 0;
  bool first_seg = true;
  bool held = false;  // a part that the CTA may join with its other warps' is still in registers
  float o[NB][MT][4], m[NB][2], l[NB][2];
  Queries<D, NB> qr;
  if (any) qr.load(a, seg, g, t);
  auto write_begun = [&](int slot) {
    if (lane != 0 || seg.u0 != 0) return;
    Begun* to = reinterpret_cast<Begun*>(r.rec) + blockIdx.x * WARPS + warp;
    *to = {slot, (int)((seg.units - seg.u1 + per - 1) / per), seg.s.q0, seg.s.n * a.group, seg.h, seg.tile};
  };
  auto write_part = [&](int slot) {
    float* part = r.part + ((size_t)(blockIdx.x * WARPS + warp) * 2 + slot) * part_floats(D, NB);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = 8 * nb + 2 * t + i;
#pragma unroll
        for (int j = 0; j < MT; j += 2)
          *reinterpret_cast<float4*>(part + row * D + 2 * MT * g + 2 * j) =
              make_float4(o[nb][j][i], o[nb][j][2 + i], o[nb][j + 1][i], o[nb][j + 1][2 + i]);
        if (g == 0) *reinterpret_cast<float2*>(part + ROWS * D + 2 * row) = make_float2(m[nb][i], l[nb][i]);
      }
    write_begun(slot);
  };
  for (bool go = any; go;) {
    Seg nxt = seg;
    go = next_seg<ROWS>(a, nxt);
    const Seq s = seg.s;
    const int rows = s.n * a.group, row0 = seg.tile * ROWS;
    // queries as fp16 scaled to [2^14, 2^15): lane (g, t) loads row 8 nb + g (its
    // operand's column) and computes with rows 8 nb + 2t and 8 nb + 2t + 1
    uint32_t qf[NB][MT][2];
    float fr[NB][2];
    int lim[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int row = row0 + 8 * nb + g;
      const bool real = row < rows;
      const int tok = real ? row / a.group : 0;
      const int sees = !real ? 0 : a.causal ? min(s.kv, s.kv - s.n + tok + 1) : s.kv;
      float f[CH][16];
      float amax = 0.f;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const uint4& y = qr.x[nb][c][v];
          const uint32_t w[4] = {y.x, y.y, y.z, y.w};
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
      const float down = a.scale_log2 * (e < 128 ? pow2f(e - 14) : 1.f);
#pragma unroll
      for (int k = 0; k < MT; ++k) {
        const float* y = &f[k / 4][4 * (k % 4)];
        qf[nb][k][0] = pack_f16(y[0] * up, y[1] * up);
        qf[nb][k][1] = pack_f16(y[2] * up, y[3] * up);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        fr[nb][i] = __shfl_sync(~0u, down, 4 * (2 * t + i));
        lim[nb][i] = __shfl_sync(~0u, sees, 4 * (2 * t + i));
      }
    }
    if (go) qr.load(a, nxt, g, t);
    const int first_lim = a.causal ? min(s.kv, s.kv - s.n + row0 / a.group + 1) : s.kv;

    // The base m of the exponents is a row's maximum when it was last raised: it is
    // raised only when a score passes it by more than P_ROOM, so most units exchange
    // no maximum and rescale nothing. A row's first score always raises it.
    float room[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      m[nb][0] = m[nb][1] = 0.f;
      room[nb][0] = room[nb][1] = NEG_INF;
      l[nb][0] = l[nb][1] = 0.f;
#pragma unroll
      for (int i = 0; i < MT; ++i) o[nb][i][0] = o[nb][i][1] = o[nb][i][2] = o[nb][i][3] = 0.f;
    }
    for (int u = seg.u0 + phase; u < seg.u1; u += STRIDE) {
      const int st = it % STAGES, j0 = u * STEP;
      if (ok) ok = __all_sync(~0u, wait_for(bars + 8 * st, (it / STAGES) & 1, abort_flag, a.status));
      if (!ok) break;
      ++it;
      const uint32_t kt = ring + st * L::STAGE, vt = kt + L::TILE;
      const float* sc = sc_sh + st * 4;
      const float ksc[2] = {sc[0], halves ? sc[2] : sc[0]};
      const float vsc[2] = {sc[1], halves ? sc[3] : sc[1]};
      // x[nb][half]: scores of tokens 16 half + rho(g) (elements 0, 1: rows 2t, 2t + 1)
      // and 16 half + 8 + rho(g) (elements 2, 3)
      float x[NB][2][4];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) x[nb][half][0] = x[nb][half][1] = x[nb][half][2] = x[nb][half][3] = 0.f;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          const uint4 lo = dec::lds128(kt + piece<D>(16 * half + rho(g), 4 * c + t));
          const uint4 hi = dec::lds128(kt + piece<D>(16 * half + 8 + rho(g), 4 * c + t));
          const uint32_t wl[4] = {lo.x, lo.y, lo.z, lo.w}, wh[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t af[4] = {
                e4m3x2_to_f16x2((uint16_t)(wl[k] & 0xFFFF)), e4m3x2_to_f16x2((uint16_t)(wh[k] & 0xFFFF)),
                e4m3x2_to_f16x2((uint16_t)(wl[k] >> 16)), e4m3x2_to_f16x2((uint16_t)(wh[k] >> 16))};
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
              mma_f16(x[nb][half], af, qf[nb][4 * c + k][0], qf[nb][4 * c + k][1]);
          }
        }
      }
      // the value codes of tokens rho(2t), rho(2t + 1) of each eight
      uint32_t vq[4][2][D / 32];
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int row = 8 * n + rho(2 * t + e);
          if constexpr (D == 128) {
            const uint4 y = dec::lds128(vt + piece<D>(row, g));
            vq[n][e][0] = y.x, vq[n][e][1] = y.y, vq[n][e][2] = y.z, vq[n][e][3] = y.w;
          } else {
            const uint2 y = lds64(vt + piece<D>(row, g >> 1) + 8 * (g & 1));
            vq[n][e][0] = y.x, vq[n][e][1] = y.y;
          }
        }
      __syncwarp();
      if (lane == 0) fence_proxy_async_smem();  // the reads of the stage precede its refill
      issue();  // into the stage just read

#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const float lv = __log2f(vsc[half]);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float f = fr[nb][i] * ksc[half], c = lv - m[nb][i] + P_UP;
            x[nb][half][i] = x[nb][half][i] * f + c;
            x[nb][half][2 + i] = x[nb][half][2 + i] * f + c;
          }
      }
      if (j0 + STEP > first_lim || ksc[0] == NEG_INF || ksc[1] == NEG_INF) {
        // Some row does not see every token. Slots that hold none leave the value
        // operand. So do NaN codes, since 0 * NaN is NaN: they come back through the
        // scores of the rows that see them.
        uint32_t nan_tokens = 0;
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int col = 8 * n + rho(2 * t + e);
            const bool in = j0 + col < s.kv && ksc[n >> 1] != NEG_INF;
#pragma unroll
            for (int w = 0; w < D / 32; ++w) {
              if (!in) vq[n][e][w] = 0;
              if (zero_nan_codes(vq[n][e][w])) nan_tokens |= 1u << col;
            }
          }
        nan_tokens = __reduce_or_sync(~0u, nan_tokens);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float& y = x[nb][n >> 1][2 * (n & 1) + i];
              const int col = 8 * n + rho(g);
              if (nan_tokens >> col & 1) y = __int_as_float(0x7FFFFFFF);
              if (j0 + col >= lim[nb][i] || ksc[n >> 1] == NEG_INF) y = NEG_INF;
            }
      }
      float top[NB][2];
      bool over = false;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          top[nb][i] = fmaxf(fmaxf(x[nb][0][i], x[nb][0][2 + i]), fmaxf(x[nb][1][i], x[nb][1][2 + i]));
          over |= top[nb][i] > room[nb][i];
        }
      if (__any_sync(~0u, over)) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float y = top[nb][i];  // relative to m - P_UP
            y = fmaxf(y, __shfl_xor_sync(~0u, y, 4));
            y = fmaxf(y, __shfl_xor_sync(~0u, y, 8));
            y = fmaxf(y, __shfl_xor_sync(~0u, y, 16));
            const bool first = room[nb][i] == NEG_INF;
            float up = 0.f, to = 0.f;
            if (y != NEG_INF && (first || y > P_UP)) {
              up = y - P_UP;
              to = P_UP;
              room[nb][i] = P_UP + P_ROOM;
            } else {
              y = 0.f;
            }
            m[nb][i] += up;
            const float f = first ? 0.f : ex2(-up);
            l[nb][i] *= f;
#pragma unroll
            for (int j = 0; j < MT; ++j) {
              o[nb][j][i] *= f;
              o[nb][j][2 + i] *= f;
            }
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              x[nb][half][i] = x[nb][half][i] - y + to;  // (y - P_UP would round large scores)
              x[nb][half][2 + i] = x[nb][half][2 + i] - y + to;
            }
          }
      }
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t pf[NB][2];
        const float iv = __fdividef(1.f, vsc[half]);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          float* y = x[nb][half];
#pragma unroll
          for (int i = 0; i < 4; ++i) y[i] = ex2(y[i]);
          l[nb][0] += (y[0] + y[2]) * iv;
          l[nb][1] += (y[1] + y[3]) * iv;
          pf[nb][0] = transpose8x8(pack_f16(y[0], y[1]));
          pf[nb][1] = transpose8x8(pack_f16(y[2], y[3]));
        }
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
          const uint32_t a0 = vq[2 * half][0][w], a1 = vq[2 * half][1][w];
          const uint32_t b0 = vq[2 * half + 1][0][w], b1 = vq[2 * half + 1][1][w];
#pragma unroll
          for (int k = 0; k < 2; ++k) {  // columns D/8 g + 4 w + 2 k and the next
            const uint32_t ap = prmt(a0, a1, k ? 0x7362 : 0x5140), bp = prmt(b0, b1, k ? 0x7362 : 0x5140);
            const uint32_t af[4] = {
                e4m3x2_to_f16x2((uint16_t)(ap & 0xFFFF)), e4m3x2_to_f16x2((uint16_t)(ap >> 16)),
                e4m3x2_to_f16x2((uint16_t)(bp & 0xFFFF)), e4m3x2_to_f16x2((uint16_t)(bp >> 16))};
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) mma_f16(o[nb][2 * w + k], af, pf[nb][0], pf[nb][1]);
          }
        }
      }
    }

    // lane (g, t) holds, of rows 2t and 2t + 1 of each eight, columns D/8 g .. D/8 (g + 1) - 1
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (room[nb][i] == NEG_INF) m[nb][i] = NEG_INF;  // saw nothing
        float& sum = l[nb][i];
        sum += __shfl_xor_sync(~0u, sum, 4);
        sum += __shfl_xor_sync(~0u, sum, 8);
        sum += __shfl_xor_sync(~0u, sum, 16);
      }
    if constexpr (!SPLIT) break;  // the item's only part
    const bool whole = seg.u0 == 0 && seg.u1 == seg.units;
    if (whole) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int rr = row0 + 8 * nb + 2 * t + i;
          if (rr >= rows) continue;
          const float inv = l[nb][i] == 0.f ? 0.f : 1.f / l[nb][i];
          uint16_t* dst = out_row<D>(a, seg, rr) + 2 * MT * g;
#pragma unroll
          for (int j = 0; j < MT; j += 4) {
            uint32_t y[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) y[k] = pack_out<BF16>(o[nb][j + k][i] * inv, o[nb][j + k][2 + i] * inv);
            *reinterpret_cast<uint4*>(dst + 2 * j) = make_uint4(y[0], y[1], y[2], y[3]);
          }
        }
    } else if (!go && first_seg) {
      held = true;
      break;
    } else {
      write_part(first_seg ? 0 : 1);
    }
    first_seg = false;
    seg = nxt;
  }

  // ---- join the warps: of an item's CTA; or, of a split call, where all four
  // hold a part of the same item and nothing else (long sequences), into one part
  bool join = true;
  if constexpr (SPLIT) {
    int* key = reinterpret_cast<int*>(smem + L::OFF_MISC + 8);  // [WARPS][4]
    __syncthreads();  // the lengths there have been read
    if (lane < 4)
      key[4 * warp + lane] = lane == 0 ? (held && ok) : lane == 1 ? seg.b : lane == 2 ? seg.h : seg.tile;
    __syncthreads();
    for (int w = 0; w < WARPS; ++w) {
      join = join && key[4 * w];
      for (int i = 1; i < 4; ++i) join = join && key[4 * w + i] == key[i];
    }
    if (held && !join) write_part(0);
  } else {
    __syncthreads();  // the rings are free
  }
  if (join) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int at = warp * ROWS + 8 * nb + 2 * t + i;
        if (g == 0) {
          m_sh[at] = m[nb][i];
          l_sh[at] = l[nb][i];
        }
        float* to = o_sh + at * L::OS + MT * 2 * g;
#pragma unroll
        for (int j = 0; j < MT; ++j)
          *reinterpret_cast<float2*>(to + 2 * j) = make_float2(o[nb][j][i], o[nb][j][2 + i]);
      }
    __syncthreads();
    constexpr int TR = THREADS / ROWS;   // threads of a row
    constexpr int TC = D / TR;           // columns of a thread, in pieces of 4 spread over the row
    const int row = threadIdx.x / TR, k = threadIdx.x % TR, rr = seg.tile * ROWS + row;
    float top = NEG_INF, sum = 0.f, acc[TC];
#pragma unroll
    for (int w = 0; w < WARPS; ++w) top = fmaxf(top, m_sh[w * ROWS + row]);
    const float base = top == NEG_INF ? 0.f : top;
#pragma unroll
    for (int n = 0; n < TC; ++n) acc[n] = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const float f = ex2(m_sh[w * ROWS + row] - base);
      const float* from = o_sh + (w * ROWS + row) * L::OS + 4 * k;
      sum += l_sh[w * ROWS + row] * f;
#pragma unroll
      for (int n = 0; n < TC; n += 2) {
        const float2 y = *reinterpret_cast<const float2*>(from + (n / 4) * 4 * TR + n % 4);
        acc[n] += y.x * f;
        acc[n + 1] += y.y * f;
      }
    }
    if constexpr (SPLIT) {
      constexpr size_t PITCH = 2 * part_floats(D, NB);
      float* p = r.part + (size_t)blockIdx.x * WARPS * PITCH;
#pragma unroll
      for (int n = 0; n < TC; n += 4)
        *reinterpret_cast<float4*>(p + row * D + n * TR + 4 * k) = make_float4(acc[n], acc[n + 1], acc[n + 2], acc[n + 3]);
      if (k < WARPS)  // the other warps' parts are in this one
        *reinterpret_cast<float2*>(p + k * PITCH + ROWS * D + 2 * row) =
            k ? make_float2(NEG_INF, 0.f) : make_float2(top, sum);
      if (warp == 0) write_begun(0);
    } else if (rr < seg.s.n * a.group) {
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      uint16_t* dst = out_row<D>(a, seg, rr) + 4 * k;
#pragma unroll
      for (int n = 0; n < TC; n += 4)
        *reinterpret_cast<uint2*>(dst + n * TR) = make_uint2(
            pack_out<BF16>(acc[n] * inv, acc[n + 1] * inv), pack_out<BF16>(acc[n + 2] * inv, acc[n + 3] * inv));
    }
  }
  if (!ok)  // gave up on a copy: let what was issued land before the memory goes
    for (int i = max(it, pit - STAGES); i < pit; ++i) drain_wait(bars + 8 * (i % STAGES), (i / STAGES) & 1);
}

// Joins one row of the items that several warps share, those begun by the four
// warps of a CTA: a warp here takes one of them, lanes its columns; where an item
// has many parts, all four take a quarter of them each. Small on purpose (its
// CTAs wait beside those of the first kernel): three reads follow one another.
constexpr int MANY = 16;  // parts

template <int D, int NB, bool BF16>
__global__ void __launch_bounds__(THREADS) join_kernel(const __grid_constant__ Rows r) {
  constexpr int V = D / 32;
  constexpr size_t PITCH = 2 * part_floats(D, NB);
  __shared__ float o_sh[WARPS][D];
  __shared__ float2 ml_sh[WARPS];
  grid_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = blockIdx.y;
  Begun it[WARPS];
  bool many = false;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    const int4* p = reinterpret_cast<const int4*>(r.rec + (blockIdx.x * WARPS + w) * 8);
    const int4 x = p[0];
    const int2 y = *reinterpret_cast<const int2*>(p + 1);
    it[w] = {x.x, x.y, x.z, x.w, y.x, y.y};
  }
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (it[w].tile * 8 * NB + row >= it[w].rows) it[w].slot = -1;
    many = many || (it[w].slot >= 0 && it[w].more >= MANY);
  }
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (it[w].slot < 0 || (!many && w != warp)) continue;
    const int worker = blockIdx.x * WARPS + w, parts = it[w].more + 1;
    const float* base0 = r.part + (size_t)worker * PITCH;
    const size_t skip = it[w].slot ? part_floats(D, NB) : 0;  // of the first part
    const int q = many ? (parts + WARPS - 1) / WARPS : parts;
    const int lo = many ? warp * q : 0, hi = min(parts, lo + q);
    float top = NEG_INF, l = 0.f, acc[V];
#pragma unroll
    for (int j = 0; j < V; ++j) acc[j] = 0.f;
    for (int i0 = lo; i0 < hi; i0 += 32) {
      const int i = i0 + lane;
      float2 ml = make_float2(NEG_INF, 0.f);
      if (i < hi) ml = *reinterpret_cast<const float2*>(base0 + i * PITCH + (i ? 0 : skip) + 8 * NB * D + 2 * row);
      float t = ml.x;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) t = fmaxf(t, __shfl_xor_sync(~0u, t, d));
      const float was = top;
      top = fmaxf(top, t);
      const float base = top == NEG_INF ? 0.f : top;
      const float back = ex2(was - base);
      // parts without tokens are not read (one that saw only NaN has an l that is not 0)
      const bool empty = ml.x == NEG_INF && ml.y == 0.f;
      const float f = empty ? 0.f : ex2(ml.x - base);
      float sum = empty ? 0.f : ml.y * f;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
      l = l * back + sum;
#pragma unroll
      for (int j = 0; j < V; ++j) acc[j] *= back;
      for (unsigned use = __ballot_sync(~0u, !empty); use;) {  // four parts' loads at a time
        float fk[4], y[4][V];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int k = use ? __ffs(use) - 1 : 0;
          fk[u] = __shfl_sync(~0u, f, k);
          if (!use) fk[u] = 0.f;
          const float* p = base0 + (i0 + k) * PITCH + (i0 + k ? 0 : skip) + row * D + V * lane;
#pragma unroll
          for (int j = 0; j < V; j += 2) {
            const float2 z = use ? *reinterpret_cast<const float2*>(p + j) : make_float2(0.f, 0.f);
            y[u][j] = z.x, y[u][j + 1] = z.y;
          }
          use &= use - 1;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int j = 0; j < V; ++j) acc[j] += y[u][j] * fk[u];
      }
    }
    if (many) {
#pragma unroll
      for (int j = 0; j < V; ++j) o_sh[warp][V * lane + j] = acc[j];
      if (lane == 0) ml_sh[warp] = make_float2(top, l);
      __syncthreads();
      top = NEG_INF;
#pragma unroll
      for (int k = 0; k < WARPS; ++k) top = fmaxf(top, ml_sh[k].x);
      const float base = top == NEG_INF ? 0.f : top;
      l = 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j) acc[j] = 0.f;
#pragma unroll
      for (int k = 0; k < WARPS; ++k) {
        const float f = ex2(ml_sh[k].x - base);
        l += ml_sh[k].y * f;
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] += o_sh[k][V * lane + j] * f;
      }
      __syncthreads();
      if (warp != 0) continue;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int rr = it[w].tile * 8 * NB + row, tok = rr / r.a.group;
    uint16_t* dst = r.a.out + ((size_t)(it[w].q0 + tok) * r.a.q_heads + it[w].h * r.a.group + (rr - tok * r.a.group)) * D;
#pragma unroll
    for (int j = 0; j < V; j += 2)
      *reinterpret_cast<uint32_t*>(dst + V * lane + j) = pack_out<BF16>(acc[j] * inv, acc[j + 1] * inv);
  }
}

// Which kernel a call runs: this one, whose 16-row tiles each read and widen the cache
// again, or that of kv8_prompt.cu. Here against there, in us, 32 heads on 8 of 128:
//   rows            16            32            48            64            80           128
//   1 x  1000  17.3 / 18.3   17.5 / 18.5   18.0 / 18.9   18.1 / 19.6   18.7 / 19.7   20.2 / 20.7
//   1 x  8000  18.4 / 19.4   19.8 / 21.6   21.2 / 25.7   23.3 / 26.6   26.2 / 27.5   34.2 / 29.6
//   1 x 64000  37.9 / 55.9   54.3 / 58.3   73.0 / 62.3   93.3 / 63.5    111 / 64.3    169 / 66.9
//  16 x  1000  20.6 / 20.9   27.3 / 21.0   32.7 / 21.4   38.6 / 21.6   43.4 / 21.7   60.7 / 22.4
//  16 x  8000  57.4 /  109   98.3 /  110    137 /  111    175 /  111    214 /  110    331 /  112
// A border of 64 suits a single sequence of some thousand tokens; batches and long
// caches would do better with 32, and a call whose sequences differ with both kernels.
bool many_rows(int max_q, int group) { return (long long)max_q * group > 64; }

bool splits(int batch, int max_kv) { return max_kv > ITEM_TOKENS && batch <= MAX_SCAN; }

// Rows of queries that share one widening of the codes, in eights.
int row_blocks(long long rows) { return rows > 8 ? 2 : 1; }

template <int D, int NB, bool BF16>
cudaError_t launch_rows(Rows& r, int sms, cudaStream_t s) {
  static bool done[2][64] = {};
  const long long rows = (long long)r.a.max_q * r.a.group;
  const long long tiles = (rows + 8 * NB - 1) / (8 * NB), items = tiles * r.a.c.heads * r.a.batch;
  cudaError_t e;
  if (!r.split) {
    constexpr int bytes = Layout<D, NB>::BYTES;
    if (items >= (1ll << 31)) return cudaErrorInvalidValue;
    r.row_tiles = (int)tiles;
    if ((e = allow_smem(rows_kernel<D, NB, BF16, false>, bytes, done[0])) != cudaSuccess) return e;
    return launch(rows_kernel<D, NB, BF16, false>, dim3((unsigned)items), THREADS, bytes, s, r);
  }
  constexpr int bytes = Layout<D, NB>::BYTES;
  if ((e = allow_smem(rows_kernel<D, NB, BF16, true>, bytes, done[1])) != cudaSuccess) return e;
  const int grid = std::min(sms, MAX_SMS) * CTAS_PER_SM;
  if ((e = launch(rows_kernel<D, NB, BF16, true>, dim3(grid), THREADS, bytes, s, r)) != cudaSuccess) return e;
  return launch(join_kernel<D, NB, BF16>, dim3(grid, (unsigned)std::min<long long>(8 * NB, rows)), THREADS, 0,
                s, r);
}

template <int D>
cudaError_t launch_d(Rows& r, int sms, cudaStream_t s) {
  if (row_blocks((long long)r.a.max_q * r.a.group) == 1)
    return r.bf16 ? launch_rows<D, 1, true>(r, sms, s) : launch_rows<D, 1, false>(r, sms, s);
  return r.bf16 ? launch_rows<D, 2, true>(r, sms, s) : launch_rows<D, 2, false>(r, sms, s);
}

}  // namespace

// Token rows of one side of the cache: [pages * heads * page][D] bytes, a box
// `rows` of them high.
bool encode_rows(CUtensorMap* map, const void* base, const Cache& c, int D, int rows) {
  auto fn = tensor_map_encoder();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)D, ((cuuint64_t)c.pages * c.heads) << c.page_shift};
  const cuuint64_t strides[1] = {(cuuint64_t)D};
  const cuuint32_t box[2] = {(cuuint32_t)D, (cuuint32_t)rows};
  const cuuint32_t estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t attention_workspace_bytes(int batch, int max_q, int max_kv, int q_heads, int kv_heads,
                                 int dim) {
  if (many_rows(max_q, q_heads / kv_heads))
    return prompt_workspace_bytes(batch, max_q, max_kv, q_heads / kv_heads, kv_heads, dim);
  if (!splits(batch, max_kv)) return 0;
  const int nb = row_blocks((long long)max_q * (q_heads / kv_heads));
  return (size_t)MAX_WORKERS * sizeof(Begun) + (size_t)MAX_WORKERS * 2 * part_floats(dim, nb) * 4;
}

cudaError_t launch_attention(const AttnArgs& a, cudaStream_t s) {
  int* status = nullptr;
  cudaError_t e = device_status_ptr(&status);
  if (e != cudaSuccess) return e;
  DeviceInfo info;
  if ((e = device_info(&info)) != cudaSuccess) return e;
  Rows r;
  r.a = {a.q, a.q_stride, a.c, a.table, a.kv_lens, a.cu_q, a.out, a.table_stride, a.batch,
         a.total_q, a.max_q, a.max_kv, a.q_heads, a.q_heads / a.c.heads, a.causal,
         a.scale * 1.44269504088896340736f, status};
  if (many_rows(a.max_q, r.a.group)) return launch_prompt(r.a, a.dim, a.bf16, a.workspace, s);
  const int box = std::min(1 << a.c.page_shift, STEP);
  if (!encode_rows(&r.tk, a.c.k, a.c, a.dim, box) || !encode_rows(&r.tv, a.c.v, a.c, a.dim, box))
    return cudaErrorInvalidValue;
  r.split = splits(a.batch, a.max_kv);
  r.bf16 = a.bf16;
  r.rec = static_cast<int*>(a.workspace);
  r.part = reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + MAX_WORKERS * sizeof(Begun));
  return a.dim == 64 ? launch_d<64>(r, info.sm_count, s) : launch_d<128>(r, info.sm_count, s);
}

}  // namespace kv8
}  // namespace w4
