// Pages of a cache: rows of a block table share them (fork), get pages of their own to write to (reserve, with
// copies of pages that others hold too), leave them (free), and the pages in use move to the front (compact).
//
// refs[p] counts the table entries that hold page p; a page with refs[p] <= 0 is free, and the lowest free pages are
// given out first, so that a call's result depends on its arguments alone.
//
// The counting is a few tens of thousands of words: one CTA does it (a grid's worth of blocks would wait for each
// other at every step), 16 loads a thread in flight, one block-wide sum for 16384 pages.  The bytes are moved by a
// kernel of the whole GPU behind it, 32 KB a block at a time, eight 16-byte loads a thread.
//
// 32 sequences of up to 32,768 positions and 16 samples of each: free 7.7 us, fork 8.1, reserve 24.4 (a chain of ten
// steps of one CTA, one to two us each) and its copies 8.1.  Room for 64 whole prompts of 32,768 positions: 95 us in pages of 64, 352 of 16 (4,096 table
// entries a round, twice).  A million rows in three caches, half of them gone: counted in 16.4 us and
// moved in 57 (177 MB in, 177 out: 6.2 TB/s).
#include <limits.h>

#include "pages.cuh"

namespace dsa {
namespace {

constexpr int kOne = 1024;         // threads of the counting CTA
constexpr int kSpan = 16;          // pages a lane looks at in a round
constexpr int kRound = kOne * kSpan;
constexpr int kItems = 4;         // table entries a thread looks at in a round
constexpr int kMove = 256;         // threads of a moving block
constexpr int kSeg = kMove * 128;  // bytes it moves at a time

__device__ __forceinline__ bool page_ok(const PagesArgs& a, int p) { return (unsigned)p < (unsigned)a.num_pages; }
__device__ __forceinline__ int64_t entry(const PagesArgs& a, int row, int j) { return row * a.ld_table + j; }

// Pages of L positions (0 <= L).
__device__ __forceinline__ int pages_of(int L, int page_size) { return L / page_size + (L % page_size != 0); }

// Exclusive sum over the block's threads of v, and the total.  (Two barriers; `part` holds a word a warp.)
__device__ __forceinline__ uint32_t block_sum(uint32_t v, uint32_t* part, uint32_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) part[warp] = x;
  __syncthreads();
  uint32_t w = part[lane];  // (the block has 32 warps)
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  const uint32_t before = warp ? __shfl_sync(0xffffffffu, w, warp - 1) : 0u;
  __syncthreads();  // part may be written again
  return before + x - v;
}

// This lane's pages of the round that starts at `base`: bit k of the answers is page base + warp · 512 + 32 k + lane.
__device__ __forceinline__ int round_page(int base, int k) {
  return base + (int)(threadIdx.x >> 5) * (32 * kSpan) + 32 * k + (int)(threadIdx.x & 31);
}

// ----------------------------------------------------------------------------
// Fork: entry i gives row dst[i] the first pages of row src[i].  A block an entry; the block looks through all entries
// for another one that writes its rows (the first entry of a row counts).
__global__ void __launch_bounds__(256) fork_kernel(const __grid_constant__ PagesArgs a) {
  griddep_wait();
  const int i = blockIdx.x;
  const int s = a.src[i], d = a.dst[i], L = a.lens[i];
  bool clash = false;
  for (int k = threadIdx.x; k < a.n; k += 256) {
    const int o = a.dst[k];
    clash |= (o == d && k < i) || o == s;
  }
  const bool ok = (unsigned)s < (unsigned)a.rows && (unsigned)d < (unsigned)a.rows && L >= 0 &&
                  L <= (int64_t)a.width * a.page_size;
  if (__syncthreads_or(clash) || !ok) {
    if (threadIdx.x == 0) atomicOr(a.status, DSA_FLAG_BAD_INDEX);
    return;
  }
  const int n = pages_of(L, a.page_size);
  for (int j = threadIdx.x; j < a.width; j += 256) {
    int p = -1;
    if (j < n) {
      p = a.table[entry(a, s, j)];
      if (page_ok(a, p)) {
        atomicAdd(a.refs + p, 1);
      } else {
        p = -1;
        atomicOr(a.status, DSA_FLAG_BAD_INDEX);
      }
    }
    a.table[entry(a, d, j)] = p;
  }
}

// Free: every entry of the row is taken once (a row may be named twice), and its page has a holder less.
__global__ void __launch_bounds__(256) free_kernel(const __grid_constant__ PagesArgs a) {
  griddep_wait();
  const int r = a.dst[blockIdx.x];
  if ((unsigned)r >= (unsigned)a.rows) {
    if (threadIdx.x == 0) atomicOr(a.status, DSA_FLAG_BAD_INDEX);
    return;
  }
  for (int j = threadIdx.x; j < a.width; j += 256) {
    const int p = atomicExch(a.table + entry(a, r, j), -1);
    if (p == -1) continue;
    if (page_ok(a, p)) {
      if (atomicSub(a.refs + p, 1) > 0) continue;
      atomicAdd(a.refs + p, 1);  // it had no holder
    }
    atomicOr(a.status, DSA_FLAG_BAD_INDEX);
  }
}

// ----------------------------------------------------------------------------
// Reserve.
struct Reserve {
  int* mark;   // [rows] the first entry of a row
  int* cnt;    // [num_pages] entries of the call that would copy a page (-1: one of them gets no pages)
  int* first;  // [num_pages] the first of them
  int* item;   // [n + 1] the table entries looked at before entry i's: its copy, if any, and those behind its held pages
  int* off;    // [n + 1] new pages before entry i's
  int* old;    // [num_pages] by new page in order: the page it replaces, -1: none, -2: not given out
  int* list;   // [num_pages] the free pages in order
  int* csrc;   // [n] what entry i copies: page, to page, rows (0: nothing); csrc is -1 for an entry that is left out,
  int* cdst;   //     -2 where nothing is copied, -3 for one that keeps a page (in cdst) which others of the call copy,
  int* crows;  //     -4 for one that was to keep it and gets nothing
  __host__ __device__ Reserve(int32_t* p, int rows, int n, int num_pages)
      : mark(p), cnt(mark + rows), first(cnt + num_pages), item(first + num_pages), off(item + n + 1), old(off + n + 1),
        list(old + num_pages), csrc(list + num_pages), cdst(csrc + n), crows(cdst + n) {}
  static int64_t words(int64_t rows, int64_t n, int64_t num_pages) { return rows + 4 * num_pages + 5 * n + 2; }
};

// A page behind the held positions that the row can keep: it is its only holder.
__device__ __forceinline__ bool own_page(const PagesArgs& a, int p) { return page_ok(a, p) && a.refs[p] == 1; }

__global__ void __launch_bounds__(kOne) reserve_kernel(const __grid_constant__ PagesArgs a) {
  griddep_wait();
  if (a.caches.n) griddep_launch();  // the moving kernel may be set up meanwhile; it waits for this one's end
  __shared__ uint32_t part[32];
  __shared__ int near[2][kOne + 1];
  Reserve R(a.scratch, a.rows, a.n, a.num_pages);
  if (a.n <= kOne) {  // (the searches below go through them ten times a thread: 3 us less for 512 entries)
    R.item = near[0];
    R.off = near[1];
  }
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, ps = a.page_size;
  // the first entry of a row counts
  for (int i = tid; i < a.n; i += kOne) {
    const int r = a.dst[i];
    if ((unsigned)r < (unsigned)a.rows) R.mark[r] = INT_MAX;
  }
  __syncthreads();
  for (int i = tid; i < a.n; i += kOne) {
    const int r = a.dst[i];
    if ((unsigned)r < (unsigned)a.rows) atomicMin(R.mark + r, i);
  }
  __syncthreads();
  for (int i = tid; i < a.n; i += kOne) {
    const int r = a.dst[i], L = a.lens[i], N = a.new_lens[i];
    bool ok = (unsigned)r < (unsigned)a.rows && L >= 0 && N >= L && N <= (int64_t)a.width * ps && R.mark[r] == i;
    int page = -2;
    if (ok && L % ps && N > L) {
      const int p = a.table[entry(a, r, L / ps)];
      ok = page_ok(a, p);  // the page of held positions is there
      if (ok && a.refs[p] > 1) {
        page = p;
        R.cnt[p] = 0;
        R.first[p] = INT_MAX;
      }
    }
    R.csrc[i] = ok ? page : -1;
    R.crows[i] = 0;
    if (!ok) {
      a.held[i] = L;
      atomicOr(a.status, DSA_FLAG_BAD_INDEX);
    }
  }
  __syncthreads();
  for (int i = tid; i < a.n; i += kOne) {
    const int p = R.csrc[i];
    if (p >= 0) {
      atomicAdd(R.cnt + p, 1);
      atomicMin(R.first + p, i);
    }
  }
  __syncthreads();
  // (a page all of whose holders are in the call stays with the first)
  uint32_t items = 0;
  for (int i0 = 0; i0 < a.n; i0 += kOne) {
    const int i = i0 + tid;
    int n = 0;
    if (i < a.n && R.csrc[i] != -1) {
      const int p = R.csrc[i];
      n = pages_of(a.new_lens[i], ps) - pages_of(a.lens[i], ps) + (p >= 0);
      if (p >= 0 && R.cnt[p] == a.refs[p] && R.first[p] == i) {
        R.csrc[i] = -3;
        R.cdst[i] = p;
        --n;
      }
    }
    uint32_t sum;
    const uint32_t before = block_sum((uint32_t)n, part, sum);
    if (i < a.n) R.item[i] = (int)(items + before);
    items += sum;  // (a table has fewer than 2^31 entries)
  }
  if (tid == 0) R.item[a.n] = (int)items;
  __syncthreads();
  // The items in the entries' order, kItems a thread side by side: which want a page, and how many did before.  visit(entry,
  // table entry's column, its page, whether it wants one, wanted before) for each; the total.
  auto walk = [&](auto visit) -> uint32_t {
    uint32_t total = 0;
    for (uint32_t x0 = 0; x0 < items; x0 += kOne * kItems) {
      const uint32_t x = x0 + tid * kItems;
      int i = 0;
      if (x < items) {
        int hi = a.n - 1;  // the last entry whose items begin at or before x
        while (i < hi) {
          const int mid = (i + hi + 1) >> 1;
          if ((uint32_t)R.item[mid] <= x) i = mid; else hi = mid - 1;
        }
      }
      int ent[kItems], col[kItems], was[kItems];
      bool need[kItems];
      uint32_t n = 0;
#pragma unroll
      for (int k = 0; k < kItems; ++k) {
        need[k] = false;
        if (x + k < items) {
          while ((uint32_t)R.item[i + 1] <= x + k) ++i;
          const bool copy = R.csrc[i] >= 0;
          const int j = (int)(x + k) - R.item[i];
          ent[k] = i;
          col[k] = copy && j == 0 ? a.lens[i] / ps : pages_of(a.lens[i], ps) + j - copy;
          was[k] = a.table[entry(a, a.dst[i], col[k])];
          need[k] = (copy && j == 0) || !own_page(a, was[k]);
          n += need[k];
        }
      }
      uint32_t sum;
      uint32_t at = total + block_sum(n, part, sum);
#pragma unroll
      for (int k = 0; k < kItems; ++k) {
        if (x + k < items) visit(ent[k], col[k], was[k], need[k], at);
        at += need[k];
      }
      total += sum;
    }
    return total;
  };
  // the new pages before each entry's (an entry without items has those of the next one with any)
  const uint32_t total = walk([&](int i, int col, int, bool, uint32_t at) {
    const int begin = R.csrc[i] >= 0 ? a.lens[i] / ps : pages_of(a.lens[i], ps);
    if (col == begin)
      for (int e = i; e >= 0 && R.item[e] == R.item[i]; --e) R.off[e] = (int)at;
  });
  __syncthreads();
  for (int i = tid; i <= a.n; i += kOne)
    if ((uint32_t)R.item[i] == items) R.off[i] = (int)total;
  // as many free pages as are wanted
  uint32_t found = 0;
  for (int64_t base = 0; base < a.num_pages && found < total; base += kRound) {
    uint32_t bits[kSpan], mine = 0;
    int v[kSpan];
#pragma unroll
    for (int k = 0; k < kSpan; ++k) {
      const int p = round_page((int)base, k);
      v[k] = p < a.num_pages ? a.refs[p] : 1;
    }
#pragma unroll
    for (int k = 0; k < kSpan; ++k) {
      bits[k] = __ballot_sync(0xffffffffu, v[k] <= 0);
      mine += __popc(bits[k]);
    }
    uint32_t sum;
    uint32_t at = block_sum(lane == 0 ? mine : 0u, part, sum);
    at = found + __shfl_sync(0xffffffffu, at, 0);
#pragma unroll
    for (int k = 0; k < kSpan; ++k) {
      if ((bits[k] >> lane) & 1u) R.list[at + __popc(bits[k] & ((1u << lane) - 1u))] = round_page((int)base, k);
      at += __popc(bits[k]);
    }
    found += sum;
  }
  __syncthreads();
  const int nfree = (int)found;
  // A page that one entry keeps and the others copy is the one's alone only if all the others get their copies: one that
  // gets nothing still holds it, and what the one wrote there would be in the other's history.
  if ((int)total > nfree) {
    for (int i = tid; i < a.n; i += kOne)
      if (R.csrc[i] >= 0 && R.off[i + 1] > nfree) R.cnt[R.csrc[i]] = -1;
    __syncthreads();
    for (int i = tid; i < a.n; i += kOne)
      if (R.csrc[i] == -3 && R.cnt[R.cdst[i]] < 0) R.csrc[i] = -4;
    __syncthreads();
  }
  auto nothing = [&](int i) { return R.off[i + 1] > nfree || R.csrc[i] == -4; };  // for entry i, if it needs pages
  // given out in the entries' order: all that an entry needs, or nothing
  for (int i = tid; i < a.n; i += kOne) {
    const int p = R.csrc[i], k0 = R.off[i], k1 = R.off[i + 1], L = a.lens[i];
    if (p == -1) continue;
    if (p == -4 || (k0 < k1 && nothing(i))) {
      a.held[i] = L;
      atomicOr(a.status, DSA_FLAG_NO_PAGES);
      continue;
    }
    a.held[i] = a.new_lens[i];
    if (p >= 0) {
      R.cdst[i] = R.list[k0];
      R.crows[i] = L % ps;
    }
  }
  walk([&](int i, int col, int was, bool need, uint32_t at) {
    if (!need || (int)at >= nfree) return;
    if (nothing(i)) {
      R.old[at] = -2;
      return;
    }
    R.old[at] = page_ok(a, was) && a.refs[was] > 1 ? was : -1;
    a.table[entry(a, a.dst[i], col)] = R.list[at];
  });
  __syncthreads();
  // the counts, which the steps above went by
  for (int k = tid; k < (int)total && k < nfree; k += kOne) {
    const int was = R.old[k];
    if (was == -2) continue;
    a.refs[R.list[k]] = 1;
    if (was >= 0) atomicSub(a.refs + was, 1);
  }
}

// ----------------------------------------------------------------------------
// Compact: the k-th page in use at or behind `live` goes to the k-th free page before it.
struct Compact {
  int* count;  // [4] moves
  int* src;    // [num_pages / 2 + 1]
  int* dst;
  __host__ __device__ Compact(int32_t* p, int num_pages) : count(p), src(p + 4), dst(src + num_pages / 2 + 1) {}
  static int64_t words(int64_t num_pages) { return 4 + 2 * (num_pages / 2 + 1); }
};

__global__ void __launch_bounds__(kOne) compact_kernel(const __grid_constant__ PagesArgs a) {
  griddep_wait();
  griddep_launch();  // (the moving kernel always follows)
  __shared__ uint32_t part[32];
  const Compact C(a.scratch, a.num_pages);
  const int tid = threadIdx.x, lane = tid & 31;
  uint32_t mine = 0, live;
  for (int64_t base = 0; base < a.num_pages; base += kRound) {
    int v[kSpan];
#pragma unroll
    for (int k = 0; k < kSpan; ++k) {
      const int p = round_page((int)base, k);
      v[k] = p < a.num_pages ? a.refs[p] : 0;
    }
#pragma unroll
    for (int k = 0; k < kSpan; ++k) mine += v[k] > 0;
  }
  block_sum(mine, part, live);
  uint32_t moves = 0, holes = 0;
  for (int64_t base = 0; base < a.num_pages; base += kRound) {
    uint32_t up[kSpan], down[kSpan], n = 0;
    int v[kSpan];
#pragma unroll
    for (int k = 0; k < kSpan; ++k) {
      const int p = round_page((int)base, k);
      v[k] = p < a.num_pages ? a.refs[p] : 0;
    }
#pragma unroll
    for (int k = 0; k < kSpan; ++k) {
      const int p = round_page((int)base, k);
      up[k] = __ballot_sync(0xffffffffu, v[k] > 0 && p >= (int)live);
      down[k] = __ballot_sync(0xffffffffu, v[k] <= 0 && p < (int)live);
      n += __popc(up[k]) | __popc(down[k]) << 16;  // (at most 16384 of each in a round)
      if (p < a.num_pages) a.moved[p] = v[k] > 0 ? p : -1;
    }
    uint32_t sum;
    uint32_t at = block_sum(lane == 0 ? n : 0u, part, sum);
    at = __shfl_sync(0xffffffffu, at, 0);
    uint32_t u = moves + (at & 0xffffu), d = holes + (at >> 16);
#pragma unroll
    for (int k = 0; k < kSpan; ++k) {
      const int p = round_page((int)base, k);
      const uint32_t below = (1u << lane) - 1u;
      if ((up[k] >> lane) & 1u) C.src[u + __popc(up[k] & below)] = p;
      if ((down[k] >> lane) & 1u) C.dst[d + __popc(down[k] & below)] = p;
      u += __popc(up[k]);
      d += __popc(down[k]);
    }
    moves += sum & 0xffffu;
    holes += sum >> 16;
  }
  __syncthreads();
  // (as many holes as moves: both are live minus those that stay)
  for (int k0 = tid; k0 < (int)moves; k0 += 8 * kOne) {
    int s[8], d[8], n[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int k = min(k0 + j * kOne, (int)moves - 1);
      s[j] = C.src[k];
      d[j] = C.dst[k];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) n[j] = a.refs[s[j]];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (k0 + j * kOne >= (int)moves) break;
      a.moved[s[j]] = d[j];
      a.refs[d[j]] = n[j];
      a.refs[s[j]] = 0;
    }
  }
  if (tid == 0) {
    C.count[0] = (int)moves;
    a.live[0] = (int)live;
  }
}

// ----------------------------------------------------------------------------
// Moving.  An item is one piece (kSeg bytes) of one cache's page; blocks take items in turn.
struct Moves {
  const int* count;  // device, or null: n
  int n;
  const int* src;
  const int* dst;
  const int* rows;   // null: whole pages
  bool remap;        // the table's entries go by a.moved first
};

__device__ __forceinline__ void move_piece(char* dst, const char* src, int bytes) {
  // pages start on 16-byte boundaries; what is left of 16 bytes at the end goes byte by byte
  constexpr int kLoads = kSeg / 16 / kMove;
  const int whole = bytes >> 4, rest = bytes & 15;
  const uint4* s = reinterpret_cast<const uint4*>(src);
  uint4* d = reinterpret_cast<uint4*>(dst);
  uint4 v[kLoads];
#pragma unroll
  for (int j = 0; j < kLoads; ++j)
    if ((int)threadIdx.x + j * kMove < whole) v[j] = __ldcs(s + threadIdx.x + j * kMove);
#pragma unroll
  for (int j = 0; j < kLoads; ++j)
    if ((int)threadIdx.x + j * kMove < whole) __stcs(d + threadIdx.x + j * kMove, v[j]);
  if ((int)threadIdx.x < rest) dst[whole * 16 + threadIdx.x] = src[whole * 16 + threadIdx.x];
}

__global__ void __launch_bounds__(kMove) move_kernel(const __grid_constant__ PagesArgs a, const Moves m) {
  griddep_wait();
  if (m.remap) {
    const int64_t all = (int64_t)a.rows * a.width;
    for (int64_t x = (int64_t)blockIdx.x * kMove + threadIdx.x; x < all; x += (int64_t)gridDim.x * kMove) {
      const int r = (int)(x / a.width);
      int32_t* e = a.table + entry(a, r, (int)(x - (int64_t)r * a.width));
      const int p = *e;
      if (p == -1) continue;
      const int to = page_ok(a, p) ? a.moved[p] : -1;
      if (to < 0) atomicOr(a.status, DSA_FLAG_BAD_INDEX);  // an entry of a page that nobody holds
      if (to != p) *e = to;
    }
  }
  const int segs = a.caches.seg0[a.caches.n];
  const int64_t items = (int64_t)(m.count ? *m.count : m.n) * segs;
  // (an item's pages are looked up while the one before it moves)
  struct Next {
    int g, rows, src, dst;
  };
  auto look = [&](int64_t x) -> Next {
    if (x >= items) return Next{0, 0, 0, 0};
    const int k = (int)(x / segs);
    return Next{(int)(x - (int64_t)k * segs), m.rows ? m.rows[k] : a.page_size, m.src[k], m.dst[k]};
  };
  Next next = look(blockIdx.x);
  for (int64_t x = blockIdx.x; x < items; x += gridDim.x) {
    const Next now = next;
    next = look(x + gridDim.x);
    if (now.rows <= 0) continue;
    int c = 0;
    while (now.g >= a.caches.seg0[c + 1]) ++c;
    const int64_t rb = a.caches.row_bytes[c], page = rb * a.page_size;
    const int64_t at = (int64_t)(now.g - a.caches.seg0[c]) * kSeg;
    const int64_t left = rb * now.rows - at;
    if (left <= 0) continue;
    char* base = a.caches.base[c];
    move_piece(base + now.dst * page + at, base + now.src * page + at, (int)(left < kSeg ? left : kSeg));
  }
}

int launch_moves(PagesArgs a, const Moves& m, int64_t most, cudaStream_t stream) {
  a.caches.seg0[0] = 0;
  for (int c = 0; c < a.caches.n; ++c)
    a.caches.seg0[c + 1] = a.caches.seg0[c] + (int)((a.caches.row_bytes[c] * a.page_size + kSeg - 1) / kSeg);
  // blocks for the most items there can be, at most what runs at once
  int64_t items = most * a.caches.seg0[a.caches.n];
  if (m.remap) {
    const int64_t blocks = ((int64_t)a.rows * a.width + kMove - 1) / kMove;
    if (blocks > items) items = blocks;
  }
  const int64_t fill = 8 * (int64_t)num_sms();
  if (items == 0) return DSA_OK;
  cudaError_t e = cudaSuccess;
  DSA_LAUNCH("move_pages", stream,
             e = launch_pdl(move_kernel, dim3((unsigned)(items < fill ? items : fill)), dim3(kMove), 0, stream, a, m));
  if (e != cudaSuccess) return set_error(DSA_ERR_CUDA, "move_pages: %s", cudaGetErrorString(e));
  return check_launch("move_pages");
}

template <typename K>
int launch_one(const char* name, K kern, int blocks, int threads, const PagesArgs& a, cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  DSA_LAUNCH(name, stream, e = launch_pdl(kern, dim3((unsigned)blocks), dim3((unsigned)threads), 0, stream, a));
  if (e != cudaSuccess) return set_error(DSA_ERR_CUDA, "%s: %s", name, cudaGetErrorString(e));
  return check_launch(name);
}

}  // namespace

size_t reserve_scratch_bytes(int rows, int n, int num_pages) { return (size_t)Reserve::words(rows, n, num_pages) * 4; }
size_t compact_scratch_bytes(int num_pages) { return (size_t)Compact::words(num_pages) * 4; }

int launch_fork_pages(const PagesArgs& a, cudaStream_t stream) { return launch_one("fork_pages", fork_kernel, a.n, 256, a, stream); }
int launch_free_pages(const PagesArgs& a, cudaStream_t stream) { return launch_one("free_pages", free_kernel, a.n, 256, a, stream); }

int launch_reserve_pages(const PagesArgs& a, cudaStream_t stream) {
  const int rc = launch_one("reserve_pages", reserve_kernel, 1, kOne, a, stream);
  if (rc != DSA_OK || a.caches.n == 0) return rc;
  const Reserve R(a.scratch, a.rows, a.n, a.num_pages);
  return launch_moves(a, Moves{nullptr, a.n, R.csrc, R.cdst, R.crows, false}, a.n, stream);
}

int launch_compact_pages(const PagesArgs& a, cudaStream_t stream) {
  const int rc = launch_one("compact_pages", compact_kernel, 1, kOne, a, stream);
  if (rc != DSA_OK) return rc;
  const Compact C(a.scratch, a.num_pages);
  return launch_moves(a, Moves{C.count, 0, C.src, C.dst, nullptr, true}, a.num_pages / 2, stream);
}

}  // namespace dsa
