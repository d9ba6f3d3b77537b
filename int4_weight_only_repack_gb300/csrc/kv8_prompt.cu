// Attention over the 8-bit cache for many rows: prompts and prompt chunks.
//
// Bound by the two products. A CTA takes 256 rows of one sequence and kv head
// (row r: token r / group, head r % group, so grouped heads fill a tile too) as
// two tiles of 128, and walks the keys in steps of 128 tokens:
//   S = Q K^T   tcgen05.mma kind::f16, both operands in shared memory
//   P = 2^(S f + log2(vs) - m + P_UP) in fp16, written over S in tensor memory
//   O += P V    A operand from tensor memory, V as stored (MN-major)
// with the two tiles half a step apart, so that one tile's products run under
// the other's exponentials. TMEM: S / P of the tiles 0-255, O 256-511.
//
// Roles (512 threads): warps 0-7 a row a thread: they scale Q to fp16, and turn S
// into P; warp 13 brings the pages' codes in by TMA, as they are, a step ahead;
// warps 8-11 widen them to fp16 (exactly) into the swizzled operand tiles, one
// layout for K (K-major) and V (MN-major); warp 12 issues the products, tile 0's
// and tile 1's in turn (issued by a warp each, the tiles fell into step and shared
// both the tensor cores and the exponentials' units); warps 14 and 15 have nothing to
// do but, in a masked call, to send for a later item's queries. Registers go where they are
// needed (setmaxnreg 184 / 184 / 96 / 48: four times the 128 of the launch).
//
// A masked call's items have the steps of the sinks and those from their first row's
// window on; which tokens a row sees is a word of 32 bits for each 32 columns, applied
// where some row of the warp does not see them all. A prompt of 8000 with a window of
// 1024 (126 GFLOP) takes 179 us; windows of 256, 512, 1536 and 2048 take 120, 141, 214 and
// 247 us, which is 1.6 us a step of an SM (8.4 steps an item at 1024) and 13.5 us an item
// around them.
//
// A CTA takes one item, the longest first (a causal sequence's last tile sees the
// most). One CTA an SM that walks a list of items, with the next item's codes and
// queries brought in under the last one's end, measured slower: 440 against 416 us
// on a prompt of 8000 tokens, 415 against 270 us on ragged chunks, since nothing
// evens out what the list deals to each. Where there are fewer than half as many
// items as SMs, an item's steps are dealt to several CTAs, whose sums a second
// kernel joins.
//
// Measured: a causal prompt of 8000 tokens, 32 heads on 8 of 128 (524 GFLOP) 415 to
// 418 us, 1260 TFLOP/s, 66 % of the cuBLAS rate. A step takes about 3250 cycles where its
// products alone are 2048, and a CTA about 9 us beyond its steps (its first codes
// and queries, the first step, the output; reading its first page numbers and
// scales before the barriers are set up is worth 2 to 6 us a call). Neither the
// exponentials nor the widening is what a step waits for: of 419 us, a build without
// the first took 399, one without the second 414. It is the chain of a tile: S, from
// tensor memory to registers and back, P V, and only behind that the next S, which is
// written where P lies. (P takes half of the columns of S; the other half, and 128
// columns where D is 64, are not used meanwhile. Half of the next S would fit there.)
// Taking the exponentials before the row's largest is known, and again in the rare
// step that raises the base, took 423 us.
//
// The base m of a row's exponents is raised only when a score passes it by more
// than P_ROOM: then its warp rescales its rows of O in tensor memory, which has to
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
using dec::drain_wait;

constexpr int TILE_ROWS = 128, CTA_ROWS = 256, KT = 128, THREADS = 512, KV_STAGES = 2;
constexpr int SOFT = 256, CONV = 128;  // threads of the roles
constexpr int TMEM_COLS = 512;
constexpr int SPLIT_SMS = 152;         // parts of items to aim at where there are few items
constexpr int SPLIT_STEPS = 16;        // that an item needs to be split
constexpr int BLK = 128 * 128;         // a block of 128 rows of 128 bytes (64 fp16 columns)
// Steps whose scales are kept. When a step's codes are brought in, the converters
// have taken those of the step before, so step - 5's rows are done with theirs.
constexpr int SLOTS = 8;

struct Prompt {
  Attn a;
  CUtensorMap tk, tv;  // token rows [pages * heads * page][D] bytes, box of a page
  int tiles;           // of the longest sequence, of CTA_ROWS rows
  int parts;           // of an item
  int sms;             // of the GPU, where the call is masked
  int bf16, mask;
  float* sums;         // with parts > 1: [item][part][D + 2][CTA_ROWS], sums, maximum, l
};

// GS: tokens that share a scale, 16 or 64 (the page's, where it has that many).
template <int D, int GS>
struct PLayout {
  static constexpr int SB = KT / GS;                       // groups of a step
  static constexpr int NB = D / 64;                        // 64-column blocks
  static constexpr int OFF_K = 2 * NB * BLK;               // after Q of both tiles
  static constexpr int OFF_V = OFF_K + KV_STAGES * NB * BLK;
  static constexpr int RAW = KT * D;                       // a step's codes
  static constexpr int OFF_RK = OFF_V + KV_STAGES * NB * BLK, OFF_RV = OFF_RK + RAW;
  static constexpr int OFF_SC = OFF_RV + RAW;              // [slot][SB] {ks, log2 vs, 1/vs, -}
  static constexpr int OFF_NAN = OFF_SC + SLOTS * SB * 16; // [slot][4] tokens with a NaN value
  static constexpr int OFF_IN = OFF_NAN + SLOTS * 16;      // [slot] sixteens that lie in a page
  static constexpr int OFF_BAR = OFF_IN + SLOTS * 4;
  static constexpr int BARS = 4 * KV_STAGES + 14;
  static constexpr int OFF_MISC = OFF_BAR + 8 * BARS;
  static constexpr int BYTES = OFF_MISC + 16 + 1024;       // + slack to align the base
  static_assert(BYTES <= 227 * 1024, "shared memory of a CTA");
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
  __device__ uint32_t qraw(int i) const { return base + 8 * (4 * KV_STAGES + 12 + i); }  // queries as they are
  __device__ uint32_t rawfull(int v) const { return base + 8 * (4 * KV_STAGES + 8 + v); }   // codes of K, V
  __device__ uint32_t rawfree(int v) const { return base + 8 * (4 * KV_STAGES + 10 + v); }
  __device__ uint32_t drained() const { return base + 8 * (4 * KV_STAGES + 7); }  // after a timeout
};

// Byte of 16-byte chunk c (of 8) of row r in a swizzled block.
__device__ __forceinline__ uint32_t sw(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }

// Shared-memory matrix descriptors with the 128-byte swizzle, as two words. The
// high one is the same for all: 8-row groups of 1024 bytes, the version, the
// swizzle. The low one has the address, in units of 16 bytes, and for V, which is
// MN-major (rows of tokens, 64 head columns a row), the stride between its
// 64-column blocks; 8-row groups are then the stride along K.
constexpr uint32_t DESC_HI = (1024 >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_kmajor(uint32_t saddr) { return (saddr >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t desc_v(uint32_t saddr) { return (saddr >> 4) | ((uint32_t)(BLK >> 4) << 16); }

// D[tmem] (+)= A * B[smem]^T, fp16 operands, A in shared or in tensor memory.
__device__ __forceinline__ void umma_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tmov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(DESC_HI)
      : "memory");
}
__device__ __forceinline__ void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tmov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(DESC_HI)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
                 "=r"(r[7])
               : "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ float half_value(uint32_t h, int bf16) {
  return bf16 ? to_float<true>((uint16_t)h) : to_float<false>((uint16_t)h);
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi, int bf16) {
  return bf16 ? pack_out<true>(lo, hi) : pack_out<false>(lo, hi);
}

// Two fp32 values in a register pair, and arithmetic on both in one instruction.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2f(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float lo2(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float hi2(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }
__device__ __forceinline__ float max3(float a, uint32_t b, uint32_t c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(__uint_as_float(b)), "f"(__uint_as_float(c)));
  return d;
}

// A score's factor, kept above zero: a masked score of -inf times it stays -inf.
__device__ __forceinline__ float factor(float fr, float ks) { return fmaxf(fr * ks, 1.17549435e-38f); }

// Two p' as fp16: a score's maximum and its exponent are rounded apart, so scores past
// 2^22 could put the largest p' beyond fp16, and it saturates there.
__device__ __forceinline__ uint32_t pack_p(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// One arrival for a warp, after all its lanes' work (each lane has put its own
// fence before it).
__device__ __forceinline__ void warp_arrive(uint32_t bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}
// One lane of a converged warp (always the same one).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Item x of a call, for a whole warp: false if there is none. `blocks` is how many its
// sequence has in each kv head, `from` the first token whose rows are its own (see below).
struct Item {
  int tile, b, h, from, blocks;
};
__device__ __forceinline__ bool bad_offsets(const Attn& a, int q0, int n) {
  return q0 < 0 || n < 0 || q0 > a.total_q - n;
}

// Item y of a kv head where offsets fall or leave 0..total_q: whoever is behind such a
// sequence may begin with rows that others before it have, and all rows counted could be
// many times those that blocks were launched for. So a row is the first sequence's that has
// it, and a sequence gets blocks for its tiles from its first own row on, one behind the
// furthest row so far. That is no more than most_tiles(): a sequence with own rows has one
// block beyond its rows' share, or two where it begins with others' rows, and before each
// of those lies one that falls and has none.
__device__ __forceinline__ bool item_among_fallen(const Prompt& p, long long y, Item& it) {
  const Attn& a = p.a;
  const int lane = threadIdx.x & 31, per = (a.batch + 31) / 32;
  const int b0 = min(a.batch, lane * per), b1 = min(a.batch, b0 + per);
  if (blockIdx.x == 0 && threadIdx.x == 0) record(a.status, W4_ERR_PAGE);
  int high = 0;  // behind the rows of this lane's sequences; then of all before them
  for (int b = b0; b < b1; ++b) {
    const int q0 = a.cu_q[b], end = a.cu_q[b + 1];
    if (!bad_offsets(a, q0, end - q0)) high = max(high, end);
  }
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int o = __shfl_up_sync(~0u, high, d);
    if (lane >= d) high = max(high, o);
  }
  high = __shfl_up_sync(~0u, high, 1);
  if (lane == 0) high = 0;
  auto blocks_of = [&](int b, int& high) {
    const int q0 = a.cu_q[b], n = a.cu_q[b + 1] - q0;
    if (bad_offsets(a, q0, n) || q0 + n <= high) return 0;
    it.from = max(q0, high) - q0;
    high = q0 + n;
    if (n > a.max_q) {  // zeros, by as many blocks as there are, or as it has rows for
      it.blocks = min(p.tiles, ((n - it.from) * a.group + CTA_ROWS - 1) / CTA_ROWS);
      it.tile = it.blocks - 1;
    } else {
      const int tiles = (n * a.group + CTA_ROWS - 1) / CTA_ROWS;
      it.blocks = tiles - it.from * a.group / CTA_ROWS;
      it.tile = tiles - 1;
    }
    return it.blocks;
  };
  long long mine = 0;
  int at = high;
  for (int b = b0; b < b1; ++b) mine += blocks_of(b, at);
  long long upto = mine;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const long long o = __shfl_up_sync(~0u, upto, d);
    if (lane >= d) upto += o;
  }
  const int owner = __ffs(__ballot_sync(~0u, y < upto)) - 1;
  if (owner < 0) return false;
  y -= __shfl_sync(~0u, upto - mine, owner);
  high = __shfl_sync(~0u, high, owner);
  int t;
  for (it.b = owner * per; (t = blocks_of(it.b, high)) <= y; ++it.b) y -= t;
  it.tile -= (int)y;
  return true;
}

// LATER: of a block that has another item now; none where offsets fall.
template <bool PACKED, bool LATER = false>
__device__ __forceinline__ bool item_at(const Prompt& p, int x, Item& it) {
  const Attn& a = p.a;
  it.from = 0, it.blocks = p.tiles;
  if (!PACKED) {  // the longest rows first: a causal sequence's last tile sees the most
    const int items = a.batch * a.c.heads, bh = x % items;
    it.tile = p.tiles - 1 - x / items, it.b = bh / a.c.heads, it.h = bh - it.b * a.c.heads;
    return true;
  }
  int y = x / a.c.heads;
  it.h = x - y * a.c.heads;
  bool fallen = false;
  auto tiles_in = [&](int b) {  // one at least, which reports a sequence that is left out
    const int q0 = a.cu_q[b], n = a.cu_q[b + 1] - q0;
    fallen |= bad_offsets(a, q0, n);
    return n > a.max_q ? p.tiles : max(1, (n * a.group + CTA_ROWS - 1) / CTA_ROWS);
  };
  const int lane = threadIdx.x & 31, per = (a.batch + 31) / 32;
  int mine = 0;  // (used where no offset falls, so that the rows are total_q at most)
#pragma unroll 4
  for (int b = lane * per; b < min(a.batch, lane * per + per); ++b) mine += tiles_in(b);
  if (__any_sync(~0u, fallen)) return !LATER && item_among_fallen(p, y, it);
  int upto = mine;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int o = __shfl_up_sync(~0u, upto, d);
    if (lane >= d) upto += o;
  }
  const int owner = __ffs(__ballot_sync(~0u, y < upto)) - 1;
  if (owner < 0) return false;
  y -= __shfl_sync(~0u, upto - mine, owner);
  int t;
  for (it.b = owner * per; (t = tiles_in(it.b)) <= y; ++it.b) y -= t;
  it.tile = t - 1 - y;
  return true;
}

// PACKED: masked and unsplit, with blocks for the tiles that the sequences have and no others.
template <int D, int GS, bool SPLIT, bool MASK, bool PACKED>
__global__ void __launch_bounds__(THREADS, 1) prompt_kernel(const __grid_constant__ Prompt p) {
  using L = PLayout<D, GS>;
  constexpr int NB = L::NB, SB = L::SB;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_addr(smem);
  const Attn& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const PBars bars{sbase + L::OFF_BAR};
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_MISC + 4);
  int* own_row = reinterpret_cast<int*>(smem + L::OFF_MISC + 8);  // with PACKED: its sequence's first

  grid_wait();
  grid_launch_dependents();
  const int parts = SPLIT ? p.parts : 1;
  const int item = blockIdx.x / parts, part = blockIdx.x - item * parts;
  Item it;
  if (!item_at<PACKED>(p, item, it)) return;
  const int tile = it.tile, b = it.b, h = it.h;
  const Seq s = load_seq(a, b);
  if (!s.ok && tid == 0 && tile == 0 && part == 0) record(a.status, W4_ERR_PAGE);
  if (s.n > a.max_q) {
    const Seq own = {s.q0 + it.from, s.n - it.from, 0, false};
    zero_rows<D>(a, own, h, tile * parts + part, it.blocks * parts);
    return;
  }
  const int rows = s.n * a.group, row0 = tile * CTA_ROWS;
  if (row0 >= rows) return;

  // tokens that a tile's last row sees, and its steps (tile 1 has the later rows)
  auto tokens_of = [&](int i) {
    const int first = row0 + TILE_ROWS * i;
    if (first >= rows) return 0;
    const int tok = (min(rows, first + TILE_ROWS) - 1) / a.group;
    return a.causal && !(MASK && a.tree) ? max(0, min(s.kv, s.kv - s.n + tok + 1)) : s.kv;
  };
  // A masked item's steps go through the sinks (whole pages and words of 32 of them) and,
  // behind them, the pages from its first row's window on: place x there is token at(x).
  // (Steps of their own for four sinks, and windows that begin with a step, were one step
  // in ten more.)
  const int first_tok = row0 / a.group, last_tok = (min(rows, row0 + CTA_ROWS) - 1) / a.group;
  const int pages_of = max(32, 1 << a.c.page_shift) - 1;
  const int sink_end = MASK ? (a.sinks + pages_of) & ~pages_of : 0;
  const int skip = MASK ? max(0, (first_seen(a, s, first_tok) >> a.c.page_shift << a.c.page_shift) - sink_end) : 0;
  auto at = [&](int x) { return MASK && x >= sink_end ? x + skip : x; };
  auto steps_of = [&](int tokens) {
    const int places = MASK && tokens > sink_end ? max(sink_end, tokens - skip) : tokens;
    return (places + KT - 1) / KT;
  };
  // this part's: steps0 and steps1 of them from step j0 on
  const int all0 = steps_of(tokens_of(0)), all1 = steps_of(tokens_of(1));
  const int per = (max(all0, all1) + parts - 1) / parts, j0 = part * per, k0 = KT * j0;
  const int steps0 = max(0, min(all0 - j0, per)), steps1 = max(0, min(all1 - j0, per));
  const int steps = max(steps0, steps1);
  auto place_of = [&](int j) { return k0 + KT * j; };  // the first of the part's step j
  // tokens from which on some row of the CTA does not see all; and, masked, until which
  const int first_lim = a.causal ? max(0, min(s.kv, s.kv - s.n + (MASK && a.tree ? 0 : first_tok + 1))) : s.kv;
  const int all_lo = MASK ? all_see_from(a, s, last_tok) : 0;
  auto partly_seen = [&](int x) {  // of the step from place x on
    if constexpr (!MASK) return x + KT > first_lim;
    // (a step with sinks and a window begins before all_lo and ends past the sinks)
    else return at(x + KT - 1) >= first_lim || (at(x) < all_lo && at(x) + KT > a.sinks);
  };

  // For the warp that brings codes in: lane g < 8 has the step's sixteen g, its page's
  // number, read two steps ahead; the first lane of a page has its copies, the first
  // of a group its scales, read a step ahead.
  const int shift = a.c.page_shift, g = lane & 7;
  const int32_t* table = a.table + (size_t)b * a.table_stride;
  const bool lead = lane < 8 && ((16 * g) & ((1 << shift) - 1)) == 0;
  const bool scales = lane < 8 && (16 * g) % GS == 0;
  const uint32_t page_bytes = (uint32_t)D << shift;
  auto page_at = [&](int j) {
    const int t = at(place_of(j) + 16 * g);
    return j < steps && t < s.kv ? table[t >> shift] : -1;
  };
  auto row_of = [&](int j, int pg) {  // page and head; -1: no page
    const bool real = j < steps && at(place_of(j) + 16 * g) < s.kv;
    if (real && (unsigned)pg >= (unsigned)a.c.pages) record(a.status, W4_ERR_PAGE);
    return real && (unsigned)pg < (unsigned)a.c.pages ? pg * a.c.heads + h : -1;
  };
  int page_row = -1, next = -1;
  float ks = 0.f, vs = 1.f;
  auto load_scales = [&]() {
    if (scales && page_row >= 0) ks = a.c.ks[page_row], vs = a.c.vs[page_row];
  };
  if (warp == 13) {  // (on their way before the barriers are ready)
    page_row = row_of(0, page_at(0)), next = page_at(1);
    load_scales();
  }

  if (tid == 0) {
    for (int i = 0; i < KV_STAGES; ++i) {
      mbar_init(bars.kfull(i), CONV / 32 + 1);  // and the scales
      mbar_init(bars.vfull(i), CONV / 32);
      mbar_init(bars.kfree(i), 1);
      mbar_init(bars.vfree(i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bars.sfull(i), 1);
      mbar_init(bars.pfull(i), SOFT / 64);
      mbar_init(bars.odone(i), 1);
      mbar_init(bars.qraw(i), TILE_ROWS);
      mbar_init(bars.rawfull(i), 1);
      mbar_init(bars.rawfree(i), CONV / 32);
    }
    mbar_init(bars.qfull(), SOFT / 32);
    mbar_init(bars.drained(), 1);
    *abort_flag = 0;
    if (PACKED) *own_row = it.from * a.group;
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

  if (warp < 8) {
    // ------------------------------------------------------------ rows: Q, then S to P
    more_registers<184>();
    const int i = warp >> 2, quarter = warp & 3;
    const int lrow = quarter * 32 + lane, row = row0 + TILE_ROWS * i + lrow;
    const bool real = row < rows && (!PACKED || row >= *own_row);
    const int tok = real ? row / a.group : 0;
    Sight sees = {0, !real ? 0 : a.causal ? min(s.kv, s.kv - s.n + tok + 1) : s.kv, 0};
    if constexpr (MASK)
      if (real) sees = sight_of(a, s, tok);
    const int my_steps = i ? steps1 : steps0;
    bool ok = true;
    float fr;
    {
      const uint16_t* src = a.q + (size_t)(s.q0 + tok) * a.q_stride +
                            (size_t)(h * a.group + (real ? row - tok * a.group : 0)) * D;
      uint4 x[D / 8];
      uint32_t most = 0;  // (magnitudes order as their bits do)
      // A thread that loads its own row touches 32 lines with its warp in each instruction,
      // and the first codes wait behind them: rows of 256 bytes are copied to their place in
      // shared memory first, where pieces are taken in turned order, so that the eight lanes
      // of a phase take them from all banks. (Window of 1024, prompt 184 -> 179 us, chunks
      // 192 -> 185; no mask, prompt 420 -> 416 us. Rows of 128 bytes lose by it: encoder
      // states 33.6 -> 35.4 us, chunks with a window 74.0 -> 75.0.)
      constexpr bool COPY = D == 128;
      uint8_t* q = smem + i * NB * BLK;
      if constexpr (COPY) {
        const uint32_t raw = smem_addr(q) + lrow * (2 * D);
        mbar_arrive_expect_tx(bars.qraw(i), 2 * D);
        dec::bulk_copy(raw, src, 2 * D, bars.qraw(i));
        ok = __all_sync(~0u, wait_for(bars.qraw(i), 0, abort_flag, a.status));
        if (!ok) drain_wait(bars.qraw(i), 0);
#pragma unroll
        for (int c = 0; c < D / 8; ++c)
          x[c] = *reinterpret_cast<const uint4*>(q + lrow * (2 * D) + 16 * ((c + lane) % (D / 8)));
        asm volatile("bar.sync %0, %1;" ::"r"(1 + i), "n"(TILE_ROWS) : "memory");  // all have taken theirs
      } else {
#pragma unroll
        for (int c = 0; c < D / 8; ++c) x[c] = *reinterpret_cast<const uint4*>(src + 8 * c);
      }
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        const uint32_t w[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) most = __vmaxu2(most, w[k] & 0x7FFF7FFFu);
      }
      const float amax = half_value(max(most & 0xFFFFu, most >> 16), p.bf16);
      // fp16 scaled to [2^14, 2^15); a negative scale goes into Q, so that fr >= 0
      const int e = max((int)(__float_as_uint(amax) >> 23) - 127, -100);
      const float up = copysignf(e < 128 ? pow2f(14 - e) : 1.f, a.scale_log2);
      fr = fabsf(a.scale_log2) * (e < 128 ? pow2f(e - 14) : 1.f);
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        const uint32_t w[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
        uint32_t y[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          y[k] = pack_f16(half_value(w[k] & 0xFFFF, p.bf16) * up, half_value(w[k] >> 16, p.bf16) * up);
        const int pc = COPY ? (c + lane) % (D / 8) : c;
        *reinterpret_cast<uint4*>(q + (pc / 8) * BLK + sw(lrow, pc % 8)) = make_uint4(y[0], y[1], y[2], y[3]);
      }
      fence_proxy_async_smem();
    }
    // A row warp sees a step's keys announced before it hands over what the products of
    // that step wait for (Q, then P of the step before): the barrier cannot go on to the
    // step after next, two phases that look alike, while a warp has yet to look.
    if (ok && my_steps > 0) ok = __all_sync(~0u, wait_for(bars.kfull(0), 0, abort_flag, a.status));
    warp_arrive(bars.qfull());
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const uint32_t st = tmem + lanes + 128 * i, ot = tmem + lanes + 256 + D * i;
    float m = 0.f, room = NEG_INF, l = 0.f;
    for (int j = 0; ok && j < my_steps; ++j) {
      ok = __all_sync(~0u, wait_for(bars.sfull(i), j & 1, abort_flag, a.status));
      if (!ok) break;
      tc_fence_after();
      uint32_t x[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(st + 32 * c, x[c]);
      const float4* sc = reinterpret_cast<const float4*>(smem + L::OFF_SC) + (j % SLOTS) * SB;
      tmem_ld_wait();
      const int x0 = place_of(j);
      if (partly_seen(x0)) {  // some row does not see every token
        const uint32_t* nan = reinterpret_cast<const uint32_t*>(smem + L::OFF_NAN) + (j % SLOTS) * 4;
        const int left = sees.lim - x0;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t bad = nan[c];
          if constexpr (MASK) {
            // (a step's mask costs what its exponentials do, so a warp applies what it needs of it)
            const int t = at(x0 + 32 * c), d = t - s.kv + s.n;  // d: the draft that the 32 tokens begin with
            uint32_t seen = below32(sees.lim - t) & (~below32(sees.lo - t) | below32(a.sinks - t));
            if (d > -32 && d < MAX_DRAFTS) seen |= (uint32_t)(d < 0 ? sees.bits << -d : sees.bits >> d);
            if (bad) {
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (bad >> k & 1) x[c][k] = 0x7FFFFFFFu;
            }
            if (!__all_sync(~0u, seen == ~0u)) {
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (!(seen >> k & 1)) x[c][k] = __float_as_uint(NEG_INF);
            }
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              if (bad >> k & 1) x[c][k] = 0x7FFFFFFFu;
              if (32 * c + k >= left) x[c][k] = __float_as_uint(NEG_INF);
            }
          }
        }
      }
      // the row's largest exponent, relative to m
      float top = NEG_INF;
#pragma unroll
      for (int g = 0; g < SB; ++g) {
        float y[4] = {NEG_INF, NEG_INF, NEG_INF, NEG_INF};
#pragma unroll
        for (int k = 0; k < GS; k += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int n = GS * g + k + 2 * e;
            y[e] = max3(y[e], x[n / 32][n % 32], x[n / 32][n % 32 + 1]);
          }
        const float4 z = sc[g];
        top = fmaxf(top, fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3])) * factor(fr, z.x) + z.y);
      }
      top -= m;
      if (__any_sync(~0u, top > room)) {
        const bool first = room == NEG_INF;
        float up = 0.f;
        if (top != NEG_INF && (first || top > 0.f)) {
          up = top;
          room = P_ROOM;
        }
        m += up;
        const float f = first ? 0.f : ex2(-up);
        l *= f;
        if (j > 0) {
          ok = __all_sync(~0u, wait_for(bars.odone(i), (j - 1) & 1, abort_flag, a.status));
          if (!ok) break;
          tc_fence_after();
          // (before a row's first score O holds zeros, which f = 0 keeps)
#pragma unroll
          for (int c = 0; c < D / 8; ++c) {  // (eight columns at a time: S stays in registers)
            uint32_t y[8];
            tmem_ld8(ot + 8 * c, y);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 8; ++k) y[k] = __float_as_uint(__uint_as_float(y[k]) * f);
            tmem_st8(ot + 8 * c, y);
          }
          tmem_st_wait();
        }
      }
      const float base = m - P_UP;
      uint64_t f2 = 0, add2 = 0, sum = 0;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t y[16];
#pragma unroll
        for (int k = 0; k < 32; k += 2) {
          const int n = 32 * c + k, g = n / GS;
          if (n % GS == 0) {
            const float4 z = sc[g];
            const float f = factor(fr, z.x), add = z.y - base;
            f2 = pack2(f, f);
            add2 = pack2(add, add);
            sum = pack2(0.f, 0.f);
          }
          const uint64_t e = fma2(pack2(__uint_as_float(x[c][k]), __uint_as_float(x[c][k + 1])), f2, add2);
          const float p0 = ex2(lo2(e)), p1 = ex2(hi2(e));
          sum = add2f(sum, pack2(p0, p1));
          y[k / 2] = pack_p(p0, p1);
          if (n % GS == GS - 2) l += (lo2(sum) + hi2(sum)) * sc[g].z;
        }
        tmem_st16(st + 16 * c, y);
      }
      if (j + 1 < my_steps)
        ok = wait_for(bars.kfull((j + 1) % KV_STAGES), ((j + 1) / KV_STAGES) & 1, abort_flag, a.status);
      tmem_st_wait();
      tc_fence_before();
      if (!(ok = __all_sync(~0u, ok))) break;
      warp_arrive(bars.pfull(i));
    }
    if (ok && my_steps > 0)
      ok = __all_sync(~0u, wait_for(bars.odone(i), (my_steps - 1) & 1, abort_flag, a.status));
    if (ok) {
      tc_fence_after();
      constexpr bool whole = !SPLIT;
      const float inv = !whole ? 1.f : l == 0.f ? 0.f : 1.f / l;
      uint16_t* dst = a.out + ((size_t)(s.q0 + tok) * a.q_heads + h * a.group + (row - tok * a.group)) * D;
      // (a column of sums at a time: a warp's rows are neighbours there)
      float* sum = whole ? nullptr : p.sums + (size_t)blockIdx.x * CTA_ROWS * (D + 2) + TILE_ROWS * i + lrow;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t y[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) y[k] = 0;
        if (my_steps > 0) {
          tmem_ld32(ot + 32 * c, y);
          tmem_ld_wait();
        }
        if (!real) continue;
#pragma unroll
        for (int k = 0; k < 32; k += 8) {
          float f[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(y[k + e]) * inv;
          if (whole) {
            *reinterpret_cast<uint4*>(dst + 32 * c + k) =
                make_uint4(pack_half(f[0], f[1], p.bf16), pack_half(f[2], f[3], p.bf16),
                           pack_half(f[4], f[5], p.bf16), pack_half(f[6], f[7], p.bf16));
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[(32 * c + k + e) * CTA_ROWS] = f[e];
          }
        }
      }
      if (!whole && real) {
        sum[D * CTA_ROWS] = room == NEG_INF ? NEG_INF : m;
        sum[(D + 1) * CTA_ROWS] = l;
      }
    }
  } else if (warp < 12) {
    // ------------------------------------------------------------ pages to operand tiles
    fewer_registers<96>();
    // A thread takes 16-byte piece p4 (+ 4 n) of row r32 (+ 32 i). Neighbouring
    // groups of four lanes take rows r and r ^ 5: the reads of a phase of eight
    // lanes then differ in bit 2 of the swizzled piece, the writes in bit 0.
    const int c = tid - SOFT, p4 = c & 3, k8 = c >> 2 & 7, cw = warp - 8;
    const int r8 = k8 & 1 ? (k8 - 1) ^ 5 : k8, r32 = 8 * cw + r8;
    uint32_t* nan = reinterpret_cast<uint32_t*>(smem + L::OFF_NAN);
    const uint32_t* in = reinterpret_cast<const uint32_t*>(smem + L::OFF_IN);
    uint4 raw[4][NB];
    auto take = [&](int at) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          const int r = 32 * i + r32;
          const int off = D == 128 ? r * 128 + (((p4 + 4 * n) ^ (r & 7)) << 4) : r * 64 + ((p4 ^ (r >> 1 & 3)) << 4);
          raw[i][n] = *reinterpret_cast<const uint4*>(smem + at + off);
        }
    };
    auto clear = [&](int i) {
#pragma unroll
      for (int n = 0; n < NB; ++n) raw[i][n] = make_uint4(0, 0, 0, 0);
    };
    auto widen = [&](int at) {
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
          *reinterpret_cast<uint4*>(smem + at + n * BLK + sw(r, 2 * p4)) = make_uint4(y[0], y[1], y[2], y[3]);
          *reinterpret_cast<uint4*>(smem + at + n * BLK + sw(r, 2 * p4 + 1)) = make_uint4(y[4], y[5], y[6], y[7]);
        }
      fence_proxy_async_smem();
    };
    auto nan_in = [&](int i) {  // clears the NaN codes of raw[i]; whether there were any
      bool hit = false;
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        hit |= zero_nan_codes(raw[i][n].x);
        hit |= zero_nan_codes(raw[i][n].y);
        hit |= zero_nan_codes(raw[i][n].z);
        hit |= zero_nan_codes(raw[i][n].w);
      }
      return hit;
    };
    // tokens of the step that are none (of a page that does not exist, or past the end)
    auto absent = [&](int j, int slot, int i) {
      const int r = 32 * i + r32;
      return !(in[slot] >> (r >> 4) & 1) || at(place_of(j) + r) >= s.kv;
    };
    auto wait_warp = [&](uint32_t bar, uint32_t ph) { return __all_sync(~0u, wait_for(bar, ph, abort_flag, a.status)); };
    for (int j = 0; j < steps; ++j) {
      const int stage = j % KV_STAGES, slot = j % SLOTS;
      const uint32_t ph = ((j / KV_STAGES) & 1) ^ 1;
      const bool edge = partly_seen(place_of(j));
      if (!wait_warp(bars.rawfull(0), j & 1)) break;
      take(L::OFF_RK);
      const bool part = at(place_of(j) + KT - 1) >= s.kv || in[slot] != 0xFFu;
      if (part) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (absent(j, slot, i)) clear(i);
      }
      fence_proxy_async_smem();  // the reads of the codes precede the copy that replaces them
      warp_arrive(bars.rawfree(0));
      if (!wait_warp(bars.kfree(stage), ph)) break;
      widen(L::OFF_K + stage * NB * BLK);
      if (edge) {
        // Some row does not see every token, and 0 * NaN is NaN: NaN values leave the
        // operand (below) and come back through the scores of the rows that see them,
        // which therefore have to know them first.
        if (!wait_warp(bars.rawfull(1), j & 1)) break;
        take(L::OFF_RV);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (part && absent(j, slot, i)) clear(i);
          // a warp has eight tokens, four lanes each: one byte of the 32 tokens' word
          uint32_t byte = __reduce_or_sync(~0u, nan_in(i) ? 1u << r8 : 0u);
          if (lane == 0) reinterpret_cast<uint8_t*>(nan)[slot * 16 + 4 * i + cw] = (uint8_t)byte;
        }
      }
      warp_arrive(bars.kfull(stage));
      if (!wait_warp(bars.rawfull(1), j & 1)) break;
      take(L::OFF_RV);
      if (edge || part) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (part && absent(j, slot, i)) clear(i);
          if (edge) nan_in(i);
        }
      }
      fence_proxy_async_smem();
      warp_arrive(bars.rawfree(1));
      if (!wait_warp(bars.vfree(stage), ph)) break;
      widen(L::OFF_V + stage * NB * BLK);
      warp_arrive(bars.vfull(stage));
    }
  } else {
    // ------------------------------------------------------------ products
    fewer_registers<48>();
    const int role = __shfl_sync(~0u, warp, 0);
    if (role == 12 && steps > 0) {
      constexpr uint32_t IDESC_S = idesc_f16(0, TILE_ROWS, KT);
      constexpr uint32_t IDESC_O = idesc_f16(0, TILE_ROWS, D) | (1u << 16);  // V is MN-major
      constexpr uint32_t TILE = NB * BLK / 16;  // a tile or stage, in the descriptors' units
      const uint32_t tm = __shfl_sync(~0u, tmem, 0);
      const uint32_t qd = desc_kmajor(sbase), kd = desc_kmajor(sbase + L::OFF_K), vd = desc_v(sbase + L::OFF_V);
      const bool leader = elect_one();
      bool ok = wait_for(bars.qfull(), 0, abort_flag, a.status), issued = false;
      auto scores = [&](int i, int j) {  // S of tile i, step j (by the leader)
        const uint32_t q = qd + i * TILE, k0 = kd + (j % KV_STAGES) * TILE;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = (k / 4) * (BLK / 16) + (k % 4) * 2;
          umma_ss(tm + 128 * i, q + off, k0 + off, IDESC_S, k != 0);
        }
      };
      auto keys = [&](int j) { return wait_for(bars.kfull(j % KV_STAGES), (j / KV_STAGES) & 1, abort_flag, a.status); };
      if ((ok = __all_sync(~0u, ok && keys(0)))) {
        tc_fence_after();
        if (leader) {
          for (int i = 0; i < 2; ++i) {
            if ((i ? steps1 : steps0) == 0) continue;
            scores(i, 0);
            umma_commit(bars.sfull(i));
          }
          umma_commit(bars.kfree(0));
        }
        issued = true;
      }
      int seen = -1;
      for (int j = 0; ok && j < steps; ++j) {
        const int stage = j % KV_STAGES;
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
          const int n = i ? steps1 : steps0;
          if (!ok || j >= n) continue;
          // O += P V of this step and S of the next, one after the other with nothing
          // waited for between: a gap there costs the tensor cores some 250 cycles
          // (the keys of a step are announced after the values of the one before)
          if (j != seen) {
            ok = j + 1 < steps ? keys(j + 1) : wait_for(bars.vfull(stage), (j / KV_STAGES) & 1, abort_flag, a.status);
            seen = j;
          }
          ok = ok && wait_for(bars.pfull(i), j & 1, abort_flag, a.status);
          if (!(ok = __all_sync(~0u, ok))) continue;
          tc_fence_after();
          if (leader) {
            const uint32_t pt = tm + 128 * i, ot = tm + 256 + D * i, v0 = vd + stage * TILE;
#pragma unroll
            for (int k = 0; k < KT / 16; ++k) umma_ts(ot, pt + 8 * k, v0 + k * 128, IDESC_O, j != 0 || k != 0);
            umma_commit(bars.odone(i));  // (first: who sees the scores has no older product to take for this one)
            if (j + 1 < n) {
              scores(i, j + 1);
              umma_commit(bars.sfull(i));
            }
            // a stage is free once the last tile that uses it has read it
            if (i == 1 || j >= steps1) umma_commit(bars.vfree(stage));
            if (j + 1 < n && (i == 1 || j + 1 >= steps1)) umma_commit(bars.kfree((j + 1) % KV_STAGES));
          }
        }
      }
      if (!ok && issued) {  // let what was issued finish before the memory goes
        if (leader) umma_commit(bars.drained());
        drain_wait(bars.drained(), 0);
      }
    } else if (role == 13 && steps > 0) {
      // ---------------------------------------------------------- codes and scales
      float4* sc = reinterpret_cast<float4*>(smem + L::OFF_SC);
      uint32_t* in = reinterpret_cast<uint32_t*>(smem + L::OFF_IN);
      bool ok = true;
      int last = -1, last_v = -1;  // steps whose copies were issued
      for (int j = 0; j < steps; ++j) {
        const int slot = j % SLOTS;
        const uint32_t ph = (j & 1) ^ 1;
        const uint32_t have = __ballot_sync(~0u, lane < 8 && page_row >= 0);
        const uint32_t bytes = __popc(__ballot_sync(~0u, lead && page_row >= 0)) * page_bytes;
        const int y = page_row << shift;  // (a step begins with a page)
        if (!(ok = __all_sync(~0u, wait_for(bars.rawfree(0), ph, abort_flag, a.status)))) break;
        if (lane == 0) {  // (what the converters read of the step comes before its barrier)
          in[slot] = have;
          mbar_arrive_expect_tx(bars.rawfull(0), bytes);
        }
        __syncwarp();
        if (lead && page_row >= 0) tma_load_2d(sbase + L::OFF_RK + 16 * g * D, &p.tk, bars.rawfull(0), 0, y);
        last = j;
        if (scales)
          sc[slot * SB + 16 * g / GS] =
              page_row < 0 ? make_float4(0.f, NEG_INF, 1.f, 0.f)
                           : make_float4(ks, __log2f(vs), __fdividef(1.f, vs), 0.f);
        warp_arrive(bars.kfull(j % KV_STAGES));
        if (!(ok = __all_sync(~0u, wait_for(bars.rawfree(1), ph, abort_flag, a.status)))) break;
        if (lane == 0) mbar_arrive_expect_tx(bars.rawfull(1), bytes);
        __syncwarp();
        if (lead && page_row >= 0) tma_load_2d(sbase + L::OFF_RV + 16 * g * D, &p.tv, bars.rawfull(1), 0, y);
        last_v = j;
        page_row = row_of(j + 1, next);
        load_scales();
        next = page_at(j + 2);
      }
      if (!ok) {  // let what was issued land before the memory goes
        if (last >= 0) drain_wait(bars.rawfull(0), last & 1);
        if (last_v >= 0) drain_wait(bars.rawfull(1), last_v & 1);
      }
    } else if (MASK && !SPLIT && role >= 14) {
      // ---------------------------------------------------------- a later item's queries, to L2
      // The item that an SM begins as it ends this one: it has nothing to do until its queries
      // are there, and an item of a window is short. (Prompt 189 -> 185 us, chunks 210 -> 206;
      // nothing gained without a mask.)
      const int later = blockIdx.x + p.sms;
      Item to;
      if (later < gridDim.x && item_at<PACKED, true>(p, later, to)) {
        const int t = to.tile, h = to.h;
        const Seq s = load_seq(a, to.b);
        for (int k = lane; k < TILE_ROWS; k += 32) {
          const int row = t * CTA_ROWS + TILE_ROWS * (role - 14) + k, tok = row / a.group;
          if (row >= s.n * a.group) break;
          const uint16_t* q = a.q + (size_t)(s.q0 + tok) * a.q_stride + (size_t)(h * a.group + row - tok * a.group) * D;
#pragma unroll
          for (int c = 0; c < D; c += 64) asm volatile("prefetch.global.L2 [%0];" ::"l"(q + c));
        }
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

// Joins the parts of 32 rows and some columns of an item that several CTAs shared. A lane
// has a row and a warp V columns, so that reads of the sums are whole lines, and AHEAD
// parts' (64 numbers a thread) are on their way before anything is done with them. The
// parts' factors come from their maxima and sums of weights: a warp takes a row there, its
// lanes the parts.
constexpr int JOIN_ROWS = 32, JOIN_WARPS = 8;
constexpr int join_cols(int d, int ahead) { return std::min(d, 64 / ahead * JOIN_WARPS); }
template <int D, int AHEAD>
__global__ void __launch_bounds__(32 * JOIN_WARPS) join_rows_kernel(const __grid_constant__ Prompt p) {
  constexpr int CW = join_cols(D, AHEAD), V = CW / JOIN_WARPS;
  __shared__ float m_sh[32][JOIN_ROWS + 1];                // a part's maximum, then its factor (-1: it saw nothing)
  __shared__ float w_sh[32][JOIN_ROWS + 1], l_sh[JOIN_ROWS];  // its sum of weights; 1 / l
  __shared__ float o_sh[JOIN_ROWS][CW + 1];
  grid_wait();
  grid_launch_dependents();
  const Attn& a = p.a;
  constexpr int COLS = D / CW, ROWS = CTA_ROWS / JOIN_ROWS;  // blocks of an item
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col0 = blockIdx.x % COLS * CW, lrow0 = blockIdx.x / COLS % ROWS * JOIN_ROWS;
  const int item = blockIdx.x / (COLS * ROWS);
  const int items = a.batch * a.c.heads, tile = p.tiles - 1 - item / items, bh = item % items;
  const int b = bh / a.c.heads, h = bh - b * a.c.heads;
  const Seq s = load_seq(a, b);
  const int row0 = tile * CTA_ROWS + lrow0, rows = min(s.n * a.group - row0, JOIN_ROWS);
  if (rows <= 0 || s.n > a.max_q) return;
  constexpr size_t PITCH = (size_t)CTA_ROWS * (D + 2);
  const float* from = p.sums + (size_t)item * p.parts * PITCH + lrow0 + lane;
  float y[AHEAD][V];
  auto ask = [&](int k0) {
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const bool take = lane < rows && k0 + k < p.parts;
#pragma unroll
      for (int e = 0; e < V; ++e) y[k][e] = take ? from[(k0 + k) * PITCH + (size_t)(col0 + V * warp + e) * CTA_ROWS] : 0.f;
    }
  };
#pragma unroll
  for (int k = 0; k < 32; k += JOIN_WARPS) {  // (at most 32 parts)
    float m = NEG_INF, l = 0.f;
    if (lane < rows && k + warp < p.parts) {
      const float* at = from + (k + warp) * PITCH + D * CTA_ROWS;
      m = at[0], l = at[CTA_ROWS];
    }
    m_sh[k + warp][lane] = m, w_sh[k + warp][lane] = l;
  }
  ask(0);
  __syncthreads();
  for (int r = warp; r < rows; r += JOIN_WARPS) {
    const float m = m_sh[lane][r], w = w_sh[lane][r];
    float top = m;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
    const float base = top == NEG_INF ? 0.f : top;
    const bool none = m == NEG_INF && w == 0.f;  // (a part that saw only NaN has an l that is not 0)
    const float f = none ? 0.f : ex2(m - base);
    float l = none ? 0.f : w * f;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(~0u, l, d);
    m_sh[lane][r] = none ? -1.f : f;
    if (lane == 0) l_sh[r] = l == 0.f ? 0.f : 1.f / l;
  }
  __syncthreads();
  if (lane < rows) {
    float o[V];
#pragma unroll
    for (int e = 0; e < V; ++e) o[e] = 0.f;
    for (int k0 = 0; k0 < p.parts; k0 += AHEAD) {
      if (k0 > 0) ask(k0);
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        const float f = m_sh[k0 + k][lane];  // (-1 where there is no part)
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] += f < 0.f ? 0.f : y[k][e] * f;
      }
    }
    const float inv = l_sh[lane];
#pragma unroll
    for (int e = 0; e < V; ++e) o_sh[lane][V * warp + e] = o[e] * inv;
  }
  __syncthreads();
  const int r = threadIdx.x / 8, row = row0 + r;
  if (r >= rows) return;
  const int tok = row / a.group;
  uint16_t* dst = a.out + ((size_t)(s.q0 + tok) * a.q_heads + h * a.group + (row - tok * a.group)) * D + col0;
#pragma unroll
  for (int c = threadIdx.x % 8 * 4; c < CW; c += 32)
    *reinterpret_cast<uint2*>(dst + c) = make_uint2(pack_half(o_sh[r][c], o_sh[r][c + 1], p.bf16),
                                                    pack_half(o_sh[r][c + 2], o_sh[r][c + 3], p.bf16));
}

// The most tiles that all sequences can have between them: one each is not full.
long long most_tiles(const Attn& a) { return (long long)a.total_q * a.group / CTA_ROWS + a.batch; }

template <int D, int GS, bool SPLIT, bool MASK, bool PACKED = false>
cudaError_t launch_it(Prompt& p, cudaStream_t s) {
  static bool done[64] = {};
  constexpr int bytes = PLayout<D, GS>::BYTES;
  cudaError_t e = allow_smem(prompt_kernel<D, GS, SPLIT, MASK, PACKED>, bytes, done);
  if (e != cudaSuccess) return e;
  const long long items = (PACKED ? most_tiles(p.a) : (long long)p.tiles * p.a.batch) * p.a.c.heads;
  const long long total = items * p.parts;
  if (total >= (1ll << 30) || !encode_rows(&p.tk, p.a.c.k, p.a.c, D, 1 << p.a.c.page_shift) ||
      !encode_rows(&p.tv, p.a.c.v, p.a.c, D, 1 << p.a.c.page_shift))
    return cudaErrorInvalidValue;
  e = launch(prompt_kernel<D, GS, SPLIT, MASK, PACKED>, dim3((unsigned)total), THREADS, bytes, s, p);
  if (e != cudaSuccess || !SPLIT) return e;
  auto join = [&](auto kernel, int ahead) {
    return launch(kernel, dim3((unsigned)(items * (CTA_ROWS / JOIN_ROWS) * (D / join_cols(D, ahead)))),
                  32 * JOIN_WARPS, 0, s, p);
  };
  return p.parts <= 4   ? join(join_rows_kernel<D, 4>, 4)
         : p.parts <= 8 ? join(join_rows_kernel<D, 8>, 8)
                        : join(join_rows_kernel<D, 16>, 16);
}

template <int D, int GS>
cudaError_t launch_parts(Prompt& p, bool packed, cudaStream_t s) {
  if (packed) return launch_it<D, GS, false, true, true>(p, s);
  if (p.mask) return p.parts > 1 ? launch_it<D, GS, true, true>(p, s) : launch_it<D, GS, false, true>(p, s);
  return p.parts > 1 ? launch_it<D, GS, true, false>(p, s) : launch_it<D, GS, false, false>(p, s);
}

// Parts of an item: enough to give every SM one, of two steps at least. Measured
// on one sequence, 8 kv heads and groups of 4, split against not: 128 queries over
// 32768 tokens 66 against 425 us, 64 over 2048 18 against 37 us; 256 over 1024 were 29
// against 25 us when a row's sums were written by its thread and joined one part after
// another (76 and 26 us above): sums in fp32 and a second launch cost some six steps.
int prompt_parts(long long items, long long max_kv) {
  const long long steps = (max_kv + KT - 1) / KT;
  if (steps < SPLIT_STEPS) return 1;
  return (int)std::max<long long>(1, std::min<long long>({SPLIT_SMS / items, steps / 2, 32}));
}

// Of a masked call, no more than `room`, which the workspace has: none without a step of
// the longest item (47 steps are 16 parts of 3, not 19); and where a window hides tokens,
// so that items are short, split only if that leaves out 6 of an item's steps, or 4 where
// the sums are few. Measured with windows on one sequence of 8000, split against not:
// groups of 4, 256 queries, a window of 1024 (10 steps, 32 items) 21.3 against 27.3 us,
// 512 (6 steps) 20.7 against 20.3; 512 queries (64 items in 2 parts), 1536 32.9 against
// 34.3, 1024 29.4 against 27.7; groups of 1, 128 queries (8 items), 512 15.7 against 19.8.
int masked_parts(long long items, int room, long long max_kv, long long seen) {
  const long long steps = (seen + KT - 1) / KT, most = std::max<long long>(1, std::min<long long>(room, steps / 2));
  const long long per = (steps + most - 1) / most, parts = (steps + per - 1) / per;
  const bool pays = seen >= max_kv || steps - per >= 6 || (steps - per >= 4 && items * parts <= 64);
  return pays ? (int)parts : 1;
}

// Sequences of different lengths leave blocks of the longest one's without a row, which
// take 0.9 us of an SM each. To find an item by all sequences' lengths takes longer the
// more there are: some 1 us for 200 of them, and twice that past 768, at each item's
// beginning. So it is found so where half of the blocks at least would be without a row, and
// those that an item is spared cost more than it. Found / by number, in us, a chunk beside
// single tokens: 2000 rows of 4 heads beside 63 of them, 8 kv heads, window of 1024 133 / 235;
// 300 beside 15 48 / 47; chunks of 100 to 2000, 20 blocks of 32 at most, 187 / 182. Groups
// of 4 on 2 kv heads of 64, sequences in all, window of 128:
//   chunk    128          256          512          768         1000         4000
//     150   15.7 / 18.1  30.9 / 33.1  65.5 / 58.7  92.8 / 85.5   218 / 109   1481 / 571
//     300   16.2 / 21.9  31.0 / 40.3  65.6 / 73.0  93.2 / 106    218 / 137
//    2000   20.0 / 67.4  32.1 / 129   68.5 / 247   95.6 / 365    223 / 472   1491 / 2001
// (16000 of them 21.7 / 2.3 ms beside 150 queries, 21.7 / 8.1 beside 2000.)
bool packing_pays(const Attn& a, int tiles) {
  const double blocks = (double)tiles * a.batch, most = (double)most_tiles(a);
  return 2 * most <= blocks && 0.9 * (blocks / most - 1) >= a.batch * (a.batch > 768 ? 0.01 : 0.005);
}

}  // namespace

size_t prompt_workspace_bytes(int batch, int max_q, int max_kv, int group, int kv_heads, int dim) {
  const long long items = ((long long)max_q * group + CTA_ROWS - 1) / CTA_ROWS * kv_heads * batch;
  const int parts = prompt_parts(items, max_kv);
  return parts > 1 ? (size_t)(items * parts) * CTA_ROWS * (dim + 2) * 4 : 0;
}

cudaError_t launch_prompt(const Attn& a, int dim, int bf16, int mask, void* workspace, cudaStream_t s) {
  Prompt p;
  p.a = a;
  p.bf16 = bf16;
  p.mask = mask;
  p.sms = 0;
  if (mask) {
    DeviceInfo info;
    const cudaError_t e = device_info(&info);
    if (e != cudaSuccess) return e;
    p.sms = info.sm_count;
  }
  p.tiles = (int)(((long long)a.max_q * a.group + CTA_ROWS - 1) / CTA_ROWS);
  const long long items = (long long)p.tiles * a.c.heads * a.batch;
  p.parts = prompt_parts(items, a.max_kv);
  if (mask && p.parts > 1) p.parts = masked_parts(items, p.parts, a.max_kv, seen_at_most(a, CTA_ROWS / a.group + 2));
  const bool packed = mask && p.parts == 1 && packing_pays(a, p.tiles);
  p.sums = static_cast<float*>(workspace);
  if (dim == 64) return a.c.page_shift >= 6 ? launch_parts<64, 64>(p, packed, s) : launch_parts<64, 16>(p, packed, s);
  return a.c.page_shift >= 6 ? launch_parts<128, 64>(p, packed, s) : launch_parts<128, 16>(p, packed, s);
}

}  // namespace kv8
}  // namespace w4
