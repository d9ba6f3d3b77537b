// Pages of the 8-bit key-value cache: reserve, fork, free, compact, copy.
//
// The reference counts are the only record of which pages are free. "The
// lowest free pages, in order" is a stream compaction of refs == 0, so the
// results never depend on the order in which threads arrive. A pool has some
// thousand to a million pages (4 MB of counts at most), too few to fill the
// GPU and bound by latency, so each call is ONE launch of one cluster of
// eight CTAs: 256 warps each take a contiguous chunk of pages and count by
// ballot, the counts are exchanged through distributed shared memory, and
// every warp then knows the rank of its pages. Only the copy of the pages
// themselves, bound by HBM, is a grid over the whole GPU. On a pool of 8000 pages
// and 100 sequences finding the moves takes 9 us and renumbering the tables 4;
// copying the 452 MB takes 74 us, 6.1 TB/s.
#include <cooperative_groups.h>

#include <algorithm>

#include "decode_common.cuh"
#include "kv8_device.cuh"

namespace w4 {
namespace kv8 {
namespace {

namespace cg = cooperative_groups;

constexpr int CL = 8;              // CTAs of the cluster (the portable maximum)
constexpr int BT = 1024;           // threads of a CTA
constexpr int BW = BT / 32;        // warps of a CTA
constexpr int NW = CL * BW;        // warps of the cluster

struct Book {
  int32_t *refs, *table, *lens;
  int pages, stride, seqs, shift;
  const int32_t *list, *list2;
  int n;
  int32_t *copy_src, *copy_dst;
  int32_t* status_out;  // or nullptr
  int* status;          // the library's device status word
  int32_t* ws;
};

// Per-warp counts of the cluster, exchanged once: [0] pages, [1] pages needed.
struct Counts {
  int own[2][BW];   // this CTA's warps
  int before[2][BW];  // what the cluster's warps before each of them counted
  int total[2];
  int err[2];       // this CTA's error, in each of two steps
};

__device__ __forceinline__ int lane_id() { return threadIdx.x & 31; }
__device__ __forceinline__ int warp_id() { return threadIdx.x >> 5; }
__device__ __forceinline__ unsigned lanes_below() { return (1u << lane_id()) - 1u; }

// The chunk [lo, hi) of n items that cluster warp w takes: whole 32s.
__device__ __forceinline__ void chunk(int n, int w, int* lo, int* hi) {
  const int per = ((n + NW - 1) / NW + 31) & ~31;
  *lo = min(n, w * per);
  *hi = min(n, *lo + per);
}

// Exchange the warps' counts: every CTA reads all 256 of both kinds (warp 0:
// pages, warp 1: needs), sums what lies before its own warps and in all. Sums stop at
// `cap`, which is more pages than there are: needs may add up to more than 31 bits.
__device__ void exchange(cg::cluster_group& cl, Counts& c, int cap) {
  cl.sync();
  const int rank = (int)cl.block_rank(), w = warp_id(), lane = lane_id();
  if (w < 2) {
    int run = 0;
    for (int r = 0; r < CL; ++r) {
      const Counts* o = cl.map_shared_rank(&c, r);
      const int v = o->own[w][lane];
      int inc = v;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int u = __shfl_up_sync(~0u, inc, d);
        if (lane >= d) inc = min(inc + u, cap);
      }
      if (r == rank) c.before[w][lane] = run + inc - v;  // (meant only where the total is below cap)
      run = min(run + __shfl_sync(~0u, inc, 31), cap);
    }
    if (lane == 0) c.total[w] = run;
  }
  __syncthreads();
}

// Whether any CTA of the cluster has seen an error in a step (the largest code wins).
__device__ int cluster_error(cg::cluster_group& cl, Counts& c, int step) {
  cl.sync();
  int e = 0;
  for (int r = 0; r < CL; ++r) e = max(e, cl.map_shared_rank(&c, r)->err[step]);
  return e;
}

__device__ void report(const Book& b, int err) {
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    if (b.status_out) *b.status_out = err;
    else if (err) record(b.status, err);
  }
}

// Count this warp's free (or live) pages into c.own[0].
template <bool LIVE>
__device__ void count_pages(const Book& b, Counts& c) {
  int lo, hi, n = 0;
  chunk(b.pages, blockIdx.x * BW + warp_id(), &lo, &hi);
#pragma unroll 4
  for (int p = lo + lane_id(); p < hi; p += 32) n += (b.refs[p] > 0) == LIVE;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) n += __shfl_xor_sync(~0u, n, d);
  if (lane_id() == 0) c.own[0][warp_id()] = n;
}

// List the first `want` free pages in order and take them (refs = 1).
__device__ void take_pages(const Book& b, const Counts& c, int32_t* fresh, int want) {
  int lo, hi;
  chunk(b.pages, blockIdx.x * BW + warp_id(), &lo, &hi);
  int rank = c.before[0][warp_id()];
  for (int base = lo; base < hi && rank < want; base += 32) {
    const int p = base + lane_id();
    const bool free = p < hi && b.refs[p] <= 0;
    const unsigned m = __ballot_sync(~0u, free);
    const int r = rank + __popc(m & lanes_below());
    if (free && r < want) {
      fresh[r] = p;
      b.refs[p] = 1;
    }
    rank += __popc(m);
  }
}

__device__ __forceinline__ int pages_of(long long tokens, int shift) {
  return (int)((tokens + (1ll << shift) - 1) >> shift);
}

__global__ void __launch_bounds__(BT) __cluster_dims__(CL, 1, 1) reserve_kernel(const Book b) {
  cg::cluster_group cl = cg::this_cluster();
  __shared__ Counts c;
  grid_wait();
  grid_launch_dependents();
  const int w = blockIdx.x * BW + warp_id(), lane = lane_id();
  if (threadIdx.x == 0) c.err[0] = c.err[1] = 0;
  __syncthreads();
  count_pages<false>(b, c);
  int lo, hi, need = 0;
  const int cap = b.pages + 1;
  chunk(b.seqs, w, &lo, &hi);
  for (int s = lo + lane; s < hi; s += 32) {
    const int held = b.lens[s], add = b.list[s];
    const long long sum = (long long)held + add;
    if (held < 0 || add < 0 || sum > MAX_KV || sum > ((long long)b.stride << b.shift))
      atomicMax(&c.err[0], W4_ERR_PAGE);
    else
      need = min(need + pages_of(sum, b.shift) - pages_of(held, b.shift), cap);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) need = min(need + __shfl_xor_sync(~0u, need, d), cap);
  if (lane == 0) c.own[1][warp_id()] = need;
  __syncthreads();
  int err = cluster_error(cl, c, 0);
  exchange(cl, c, cap);
  const int want = c.total[1];
  if (!err && want > c.total[0]) err = W4_ERR_NO_PAGES;
  report(b, err);
  if (!err) take_pages(b, c, b.ws, want);
  cl.sync();  // the list is complete (and no CTA leaves while its counts are read)
  if (err) return;
  int off = c.before[1][warp_id()];
  for (int base = lo; base < hi; base += 32) {
    const int s = base + lane;
    int have = 0, n = 0;
    if (s < hi) {
      const int held = b.lens[s], add = b.list[s];
      have = pages_of(held, b.shift);
      n = pages_of((long long)held + add, b.shift) - have;
      if (add) b.lens[s] = held + add;
    }
    unsigned todo = __ballot_sync(~0u, n > 0);
    while (todo) {  // the warp writes one sequence's new pages at a time
      const int l = __ffs(todo) - 1;
      todo &= todo - 1;
      const int m = __shfl_sync(~0u, n, l), at = __shfl_sync(~0u, have, l);
      int32_t* row = b.table + (size_t)(base + l) * b.stride + at;
      for (int j = lane; j < m; j += 32) row[j] = b.ws[off + j];
      off += m;
    }
  }
}

// The sequence whose tokens pair i's target gets, NONE or BAD. Targets are claimed: the
// length of pair j's is -(j + 1). A source that an earlier pair makes has what that
// pair copies; one that a later pair makes, or this one, is still empty.
constexpr int NONE = -1, BAD = -2;
__device__ __forceinline__ int root_of(const Book& b, int i) {
  for (;;) {
    const int s = b.list[i], claim = b.lens[s];
    if (claim >= 0) return s;
    const int j = -(claim + 1);
    if (j >= b.n || b.list2[j] != s) return BAD;  // no claim, but a length below zero
    if (j >= i) return NONE;
    i = j;
  }
}

__global__ void __launch_bounds__(BT) __cluster_dims__(CL, 1, 1) fork_kernel(const Book b) {
  cg::cluster_group cl = cg::this_cluster();
  __shared__ Counts c;
  grid_wait();
  grid_launch_dependents();
  int32_t* fresh = b.ws;
  int32_t* offs = b.ws + b.pages;  // per pair: whether it has claimed its target; then the
                                   // rank of its fresh page, -1 for none
  int32_t* held = offs + b.n;      // per pair: the source's tokens
  int32_t* root = b.copy_src;      // per pair, until the copies are listed there
  const int w = blockIdx.x * BW + warp_id(), lane = lane_id();
  if (threadIdx.x == 0) c.err[0] = c.err[1] = 0;
  __syncthreads();
  count_pages<false>(b, c);
  int lo, hi;
  chunk(b.n, w, &lo, &hi);
  // claim the targets: each must be empty, and only one pair's
  for (int i = lo + lane; i < hi; i += 32) {
    const int s = b.list[i], d = b.list2[i];
    const bool ok = s >= 0 && s < b.seqs && d >= 0 && d < b.seqs && atomicCAS(&b.lens[d], 0, -(i + 1)) == 0;
    offs[i] = ok;
    if (!ok) atomicMax(&c.err[0], W4_ERR_SEQ);
  }
  __syncthreads();
  int err = cluster_error(cl, c, 0);
  const bool claimed = !err;  // every target
  int want = 0;
  if (!err) {
    int need = 0;
    for (int base = lo; base < hi; base += 32) {
      const int i = base + lane;
      int part = 0;
      if (i < hi) {
        root[i] = root_of(b, i);
        int toks = root[i] < 0 ? 0 : b.lens[root[i]];
        if (root[i] == BAD || toks > ((long long)b.stride << b.shift)) {
          atomicMax(&c.err[1], W4_ERR_PAGE);
          toks = 0;
        }
        part = (toks & ((1 << b.shift) - 1)) != 0;
        held[i] = toks;
      }
      const unsigned m = __ballot_sync(~0u, part != 0);
      if (i < hi) offs[i] = part ? need + __popc(m & lanes_below()) : -1;  // + the warp's own start
      need += __popc(m);
    }
    if (lane == 0) c.own[1][warp_id()] = need;
    // the sources' page numbers, one warp a pair
    for (int i = w; i < b.n; i += NW) {
      const int s = root_of(b, i);
      if (s < 0) continue;
      const int n = min(pages_of(b.lens[s], b.shift), b.stride);
      for (int j = lane; j < n; j += 32) {
        const int p = b.table[(size_t)s * b.stride + j];
        if (p < 0 || p >= b.pages) atomicMax(&c.err[1], W4_ERR_PAGE);
      }
    }
    __syncthreads();
    err = cluster_error(cl, c, 1);
    exchange(cl, c, b.pages + 1);
    want = c.total[1];
    if (!err && want > c.total[0]) err = W4_ERR_NO_PAGES;
  }
  report(b, err);
  if (!err) {
    take_pages(b, c, fresh, want);
    for (int i = lo + lane; i < hi; i += 32)
      if (offs[i] >= 0) offs[i] += c.before[1][warp_id()];
  }
  cl.sync();
  if (err) {  // nothing is claimed or to be copied, whatever the lists held
    for (int i = lo + lane; i < hi; i += 32) {
      if (claimed || offs[i]) b.lens[b.list2[i]] = 0;
      b.copy_src[i] = b.copy_dst[i] = -1;
    }
    return;
  }
  for (int i = w; i < b.n; i += NW) {  // one warp a pair
    const int s = root[i], d = b.list2[i], toks = held[i], off = offs[i];
    const int full = toks >> b.shift;
    const int32_t* from = b.table + (size_t)max(s, 0) * b.stride;
    int32_t* to = b.table + (size_t)d * b.stride;
    const int page = off >= 0 ? fresh[off] : -1;
    const int last = off >= 0 ? from[full] : -1;
    for (int j = lane; j < b.stride; j += 32) {
      int p = -1;
      if (j < full) {
        p = from[j];
        atomicAdd(&b.refs[p], 1);
      } else if (j == full) {
        p = page;
      }
      to[j] = p;
    }
    __syncwarp();
    if (lane == 0) {
      b.lens[d] = toks;
      b.copy_src[i] = last;
      b.copy_dst[i] = page;
    }
  }
}

// One CTA a listed sequence. The exchange of its length decides which of two
// entries of the same sequence ends it, so its pages drop by one exactly once.
__global__ void __launch_bounds__(128) free_kernel(const Book b) {
  __shared__ int toks_sh;
  grid_wait();
  grid_launch_dependents();
  int* status = b.status_out ? b.status_out : b.status;
  const int s = b.list[blockIdx.x];
  if (s < 0 || s >= b.seqs) {
    if (threadIdx.x == 0) record(status, W4_ERR_SEQ);
    return;
  }
  if (threadIdx.x == 0) toks_sh = atomicExch(&b.lens[s], 0);
  __syncthreads();
  const long long toks = toks_sh;
  if (toks == 0) return;
  if (toks < 0 || toks > ((long long)b.stride << b.shift)) {  // no length: left as it was
    if (threadIdx.x == 0) {
      b.lens[s] = toks_sh;
      record(status, W4_ERR_PAGE);
    }
    return;
  }
  const int n = pages_of(toks, b.shift);
  int32_t* row = b.table + (size_t)s * b.stride;
  for (int j = threadIdx.x; j < b.stride; j += blockDim.x) {
    const int p = row[j];
    row[j] = -1;
    if (j >= n) continue;
    if (p < 0 || p >= b.pages) {
      record(status, W4_ERR_PAGE);
    } else if (atomicSub(&b.refs[p], 1) <= 0) {  // it was free already: leave it so
      atomicAdd(&b.refs[p], 1);
      record(status, W4_ERR_PAGE);
    }
  }
}

__global__ void clear_status_kernel(int32_t* status) {
  grid_wait();
  grid_launch_dependents();
  *status = W4_OK;
}

// ws: [0] pages in use, [16 + p] the page that p becomes (p at or above that number).
constexpr int MAP_AT = 16;

__global__ void __launch_bounds__(BT) __cluster_dims__(CL, 1, 1) compact_kernel(const Book b) {
  cg::cluster_group cl = cg::this_cluster();
  __shared__ Counts c;
  __shared__ int holes_sh;
  grid_wait();
  grid_launch_dependents();
  const int w = blockIdx.x * BW + warp_id(), lane = lane_id();
  if (lane == 0) c.own[1][warp_id()] = 0;
  if (threadIdx.x == 0) holes_sh = 0;
  count_pages<true>(b, c);
  __syncthreads();
  exchange(cl, c, b.pages + 1);
  const int used = c.total[0];
  int lo, hi;
  chunk(b.pages, w, &lo, &hi);
  int n = c.before[0][warp_id()];  // live pages before this chunk
  // holes: free pages below `used`. Whoever has page `used` in its chunk knows
  // how many live ones lie below it (with used == pages there are none).
  if (used >= lo && used < hi) {
    int k = 0;
    for (int p = lo + lane; p < used; p += 32) k += b.refs[p] > 0;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) k += __shfl_xor_sync(~0u, k, d);
    if (lane < CL) *cl.map_shared_rank(&holes_sh, lane) = used - (n + k);
  }
  cl.sync();
  const int holes = holes_sh;
  for (int base = lo; base < hi; base += 32) {
    const int p = base + lane;
    const bool live = p < hi && b.refs[p] > 0;
    const unsigned m = __ballot_sync(~0u, live);
    const int before = n + __popc(m & lanes_below());
    if (p < hi) {
      if (p < used) {
        if (!live) b.copy_dst[p - before] = p;
      } else {
        b.ws[MAP_AT + p] = p;
        if (live) b.copy_src[before - (used - holes)] = p;
      }
    }
    n += __popc(m);
  }
  const int at = blockIdx.x * BT + threadIdx.x;
  for (int i = holes + at; i < b.pages; i += CL * BT) b.copy_src[i] = b.copy_dst[i] = -1;
  if (at == 0) b.ws[0] = used;
  cl.sync();
  for (int i = at; i < holes; i += CL * BT) {
    const int s = b.copy_src[i], d = b.copy_dst[i];
    b.refs[d] = b.refs[s];
    b.refs[s] = 0;
    b.ws[MAP_AT + s] = d;
  }
}

__global__ void __launch_bounds__(256) retable_kernel(int32_t* table, size_t entries,
                                                      const int32_t* ws, int pages) {
  grid_wait();
  grid_launch_dependents();
  const int used = ws[0];
  for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < entries; i += (size_t)gridDim.x * 256) {
    const int p = table[i];
    if (p >= used && p < pages) table[i] = ws[MAP_AT + p];
  }
}

// One page's codes are one run in memory (keys and values each), moved in pieces of
// 16 KB through shared memory with bulk copies both ways by one thread, five loads
// ahead of the stores. A unit of work is a page or, where the list is short, a
// share of its pieces; a CTA's units are read 128 at a time, all threads one each,
// so the -1 entries at a list's end cost one read for all of them (read one by one
// they took longer than the copy: 452 MB in 97 us with 16-byte loads and stores,
// 130 us with bulk copies, 74 us so).
constexpr int CT = 128, PIECE = 16384, RING = 6;
constexpr int COPY_SMEM = RING * PIECE + 8 * RING + 128;

__global__ void __launch_bounds__(CT) copy_kernel(const Cache c, size_t page_bytes,
                                                  const int32_t* src, const int32_t* dst, int n,
                                                  int pieces, int parts, int* status) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
  const uint32_t bars = sm100::smem_addr(smem + RING * PIECE);
  __shared__ int3 list[CT];  // source, destination, part
  __shared__ int count;
  grid_wait();
  grid_launch_dependents();
  if (threadIdx.x == 0) {
    for (int i = 0; i < RING; ++i) sm100::mbar_init(bars + 8 * i, 1);
    sm100::fence_mbar_init();
  }
  const long long units = (long long)n * parts;
  const int per = (2 * pieces + parts - 1) / parts;  // pieces (of either side) of a part
  int loads = 0, stores = 0;
  bool ok = true;
  for (long long u0 = blockIdx.x; u0 < units; u0 += (long long)gridDim.x * CT) {
    if (threadIdx.x == 0) count = 0;
    __syncthreads();
    const long long u = u0 + (long long)threadIdx.x * gridDim.x;
    if (u < units) {
      const int i = (int)(u / parts), part = (int)(u - (long long)i * parts);
      const int s = src[i], d = dst[i];
      if (s >= 0 && d >= 0) {
        if (s < c.pages && d < c.pages) list[atomicAdd(&count, 1)] = make_int3(s, d, part);
        else record(status, W4_ERR_PAGE);
      }
    }
    __syncthreads();
    const int m = count;  // (in any order: the copies do not depend on one another)
    if (threadIdx.x >= 32) {
      // the scales, a warp a page
      for (int i = (threadIdx.x >> 5) - 1; i < m; i += CT / 32 - 1) {
        const int3 e = list[i];
        if (e.z != 0) continue;
        for (int h = threadIdx.x & 31; h < c.heads; h += 32) {
          c.ks[(size_t)e.y * c.heads + h] = c.ks[(size_t)e.x * c.heads + h];
          c.vs[(size_t)e.y * c.heads + h] = c.vs[(size_t)e.x * c.heads + h];
        }
      }
    } else if (threadIdx.x == 0) {
      const int total = m * per, first = loads;
      auto where = [&](int k, size_t* off, uint8_t** base, uint32_t* bytes) {  // piece k of the list
        const int3 e = list[k / per];
        const int r = e.z * per + k % per;  // piece r >> 1 of side r & 1
        *off = (size_t)(r >> 1) * PIECE;
        *base = (r & 1) ? c.v : c.k;
        *bytes = r < 2 * pieces ? (uint32_t)min((size_t)PIECE, page_bytes - *off) : 0;
        return e;
      };
      size_t off;
      uint8_t* base;
      uint32_t bytes;
      while (ok && stores - first < total) {
        // five pieces on their way; a slot is free when its last store has read it
        while (loads - first < total && loads - stores < RING - 1) {
          const int3 e = where(loads - first, &off, &base, &bytes);
          const uint32_t bar = bars + 8 * (loads % RING);
          asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
          sm100::mbar_arrive_expect_tx(bar, bytes);
          if (bytes)
            dec::bulk_copy(sm100::smem_addr(smem + (loads % RING) * PIECE), base + e.x * page_bytes + off, bytes, bar);
          ++loads;
        }
        const int slot = stores % RING;
        const int3 e = where(stores - first, &off, &base, &bytes);
        const uint64_t t0 = sm100::globaltimer_ns();
        while (ok && !sm100::mbar_try_wait(bars + 8 * slot, (stores / RING) & 1))
          ok = sm100::globaltimer_ns() - t0 <= dec::WAIT_LIMIT_NS;
        if (!ok) {
          record(status, W4_ERR_TIMEOUT);
          for (int i = stores; i < loads; ++i) dec::drain_wait(bars + 8 * (i % RING), (i / RING) & 1);
          break;
        }
        if (bytes)
          asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(
                           base + e.y * page_bytes + off),
                       "r"(sm100::smem_addr(smem + slot * PIECE)), "r"(bytes)
                       : "memory");
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        ++stores;
      }
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

Book book(const BookArgs& a, int* status) {
  return {a.refs, a.table, a.lens, a.pages, a.table_stride, a.seqs, a.page_shift, a.list, a.list2,
          a.n, a.copy_src, a.copy_dst, a.status_out, status, static_cast<int32_t*>(a.workspace)};
}

}  // namespace

size_t pages_workspace_bytes(int num_pages, int n) {
  return ((size_t)num_pages + 2 * (size_t)n + 64) * 4;
}

cudaError_t launch_reserve(const BookArgs& a, cudaStream_t s) {
  int* status = nullptr;
  cudaError_t e = device_status_ptr(&status);
  if (e != cudaSuccess) return e;
  return launch(reserve_kernel, dim3(CL), BT, 0, s, book(a, status));
}

cudaError_t launch_fork(const BookArgs& a, cudaStream_t s) {
  int* status = nullptr;
  cudaError_t e = device_status_ptr(&status);
  if (e != cudaSuccess) return e;
  return launch(fork_kernel, dim3(CL), BT, 0, s, book(a, status));
}

cudaError_t launch_free(const BookArgs& a, cudaStream_t s) {
  int* status = nullptr;
  cudaError_t e = device_status_ptr(&status);
  if (e != cudaSuccess) return e;
  if (a.status_out && (e = launch(clear_status_kernel, dim3(1), 1, 0, s, a.status_out)) != cudaSuccess)
    return e;
  if (a.n == 0) return cudaSuccess;
  return launch(free_kernel, dim3(a.n), 128, 0, s, book(a, status));
}

cudaError_t launch_compact(const BookArgs& a, cudaStream_t s) {
  cudaError_t e = launch(compact_kernel, dim3(CL), BT, 0, s, book(a, nullptr));
  if (e != cudaSuccess || a.seqs == 0) return e;
  DeviceInfo info;
  if ((e = device_info(&info)) != cudaSuccess) return e;
  const size_t entries = (size_t)a.seqs * a.table_stride;
  const int grid = (int)std::min<size_t>((entries + 255) / 256, (size_t)info.sm_count * 8);
  return launch(retable_kernel, dim3(grid), 256, 0, s, a.table, entries,
                static_cast<const int32_t*>(a.workspace), a.pages);
}

cudaError_t launch_copy_pages(const Cache& c, int dim, const int32_t* src, const int32_t* dst,
                              int n, cudaStream_t s) {
  int* status = nullptr;
  cudaError_t e = device_status_ptr(&status);
  if (e != cudaSuccess) return e;
  DeviceInfo info;
  if ((e = device_info(&info)) != cudaSuccess) return e;
  const size_t page_bytes = ((size_t)c.heads * dim) << c.page_shift;
  const int pieces = (int)((page_bytes + PIECE - 1) / PIECE);
  const int most = info.sm_count * 2;
  const int parts = std::max(1, std::min(2 * pieces, most / n));
  const int grid = (int)std::min<long long>((long long)n * parts, most);
  static bool done[64] = {};
  if ((e = allow_smem(copy_kernel, COPY_SMEM, done)) != cudaSuccess) return e;
  return launch(copy_kernel, dim3(grid), CT, COPY_SMEM, s, c, page_bytes, src, dst, n, pieces, parts, status);
}

}  // namespace kv8
}  // namespace w4
