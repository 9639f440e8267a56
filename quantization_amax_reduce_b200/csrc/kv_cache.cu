// The paged KV cache around its attention (kv_tree.cu): page assignment with
// the slot map of a step's new tokens, the cache write (E4M3 cast or bf16
// copy), and the move of an accepted draft path to the sequence's tail.
//
// A cache is [pages, page_size, heads, 128] with the channel contiguous and
// any strides in between (token-major or head-major pages); slot s is row
// s % page_size of page s / page_size.
#include <cuda_runtime.h>

#include "kernels.h"
#include "sm100_ptx.cuh"
#include "state.cuh"

namespace fp8attn {

namespace {

__device__ __forceinline__ void raise_error(int32_t* err, uint32_t bits) {
  if (err) atomicOr(reinterpret_cast<unsigned int*>(err), bits);
}

// ---------------------------------------------------------------------------
// Page assignment
//
// want_b = ceil(seq_b / page); a row that holds more drops its last pages, a
// row that holds fewer wants new ones.  Dropped and wanted pages are ranked in
// (row, page) order; wanted rank k takes dropped rank k while there is one,
// then the free list from its end; what was dropped and not wanted goes back
// to the free list, rank reversed, so that taking pages and giving the same
// ones back leaves the list as it was.
//
// Every CTA scans the rows itself (three prefix sums, kept in shared memory:
// a few thousand 4-byte loads that hit L2) instead of a scan launch of its
// own, then the tokens and the moved pages are split over the grid.  All CTAs
// read the old state: the pages that a row holds, the dropped entries and the
// free list below its count are not written, and `owned` and the pool's count
// are committed by the CTA that finishes last (pool[1] counts; no CTA waits).
// Bound: launch and latency.  64 requests, one new token each: 7 us; 1500
// requests admitted with 8 x 10^5 tokens, and let go: 10 us each (12 bytes
// written a token are 1.5 us of HBM).  Four neighbouring tokens or pages a
// thread share their search for a row: one a thread took 24 us for 1500
// requests let go.
// ---------------------------------------------------------------------------

constexpr int kPagesThreads = 512;
constexpr int kTokensPerThread = 4;   // neighbours share the search for their row
constexpr int kPagesPerThread = 4;

struct PagesArgs {
  const int32_t* seq;
  const int32_t* fresh;
  int32_t* tables;
  int64_t table_stride;
  int width;
  int32_t* owned;
  int32_t* free_pages;
  int num_pages;
  int32_t* pool;
  int rows;
  int page_log2;
  int max_tokens;
  int32_t* cu;
  int64_t* slots;
  int32_t* positions;
  int32_t* err;
};

// Largest b with prefix[b] <= x, for prefix[0] = 0 <= x < prefix[rows].
__device__ __forceinline__ int row_of(const int32_t* prefix, int rows, int x) {
  int lo = 0, hi = rows - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (prefix[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Exclusive scan over the CTA's threads of three 64-bit values (`v` becomes
// the sum of the lower threads' values, `total` the sum of all).
__device__ void scan3(int64_t (&v)[3], int64_t (&total)[3], int64_t (*warp_sums)[3]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t own[3];
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    own[i] = v[i];
#pragma unroll
    for (int off = 1; off < 32; off *= 2) {
      const int64_t up = __shfl_up_sync(0xffffffffu, v[i], off);
      if (lane >= off) v[i] += up;
    }
    if (lane == 31) warp_sums[warp][i] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    int64_t before = 0, all = 0;
    for (int w = 0; w < kPagesThreads / 32; ++w) {
      const int64_t s = warp_sums[w][i];
      if (w < warp) before += s;
      all += s;
    }
    v[i] = before + v[i] - own[i];
    total[i] = all;
  }
}

__global__ void __launch_bounds__(kPagesThreads) assign_pages_kernel(const PagesArgs a) {
  extern __shared__ int32_t prefix[];
  __shared__ int64_t warp_sums[kPagesThreads / 32][3];
  __shared__ int s_last;
  int32_t* s_cu = prefix;                    // new tokens before a row
  int32_t* s_grow = s_cu + a.rows + 1;       // wanted pages before a row
  int32_t* s_drop = s_grow + a.rows + 1;     // dropped pages before a row
  const int page_mask = (1 << a.page_log2) - 1;
  const int64_t most = static_cast<int64_t>(a.width) << a.page_log2;

  // this thread's rows: [first, last)
  const int per = (a.rows + kPagesThreads - 1) / kPagesThreads;
  const int first = min(a.rows, static_cast<int>(threadIdx.x) * per);
  const int last = min(a.rows, first + per);
  uint32_t bad = 0;
  int64_t sum[3] = {0, 0, 0}, total[3];
  for (int b = first; b < last; ++b) {
    const int64_t seq = a.seq[b], fresh = a.fresh[b], owned = a.owned[b];
    if (fresh < 0 || fresh > seq || seq > most || owned < 0 || owned > a.width) {
      bad |= kErrSeqlens;
      continue;
    }
    const int64_t want = (seq + page_mask) >> a.page_log2;
    sum[0] += fresh;
    sum[1] += max(want - owned, int64_t{0});
    sum[2] += max(owned - want, int64_t{0});
  }
  scan3(sum, total, warp_sums);
  const int count = a.pool[0];
  if (total[0] > a.max_tokens) bad |= kErrSeqlens;
  if (count < 0 || count + total[2] > a.num_pages || total[1] > count + total[2]) bad |= kErrPages;
  const bool refused = __syncthreads_or(bad != 0) != 0;
  if (bad && blockIdx.x == 0) raise_error(a.err, bad);
  if (!refused) {
    for (int b = first; b < last; ++b) {
      const int seq = a.seq[b], owned = a.owned[b];
      const int want = static_cast<int>((static_cast<int64_t>(seq) + page_mask) >> a.page_log2);
      s_cu[b] = static_cast<int>(sum[0]);
      s_grow[b] = static_cast<int>(sum[1]);
      s_drop[b] = static_cast<int>(sum[2]);
      sum[0] += a.fresh[b];
      sum[1] += max(want - owned, 0);
      sum[2] += max(owned - want, 0);
    }
    if (threadIdx.x == 0) {
      s_cu[a.rows] = static_cast<int>(total[0]);
      s_grow[a.rows] = static_cast<int>(total[1]);
      s_drop[a.rows] = static_cast<int>(total[2]);
    }
  }
  __syncthreads();
  const int tokens = refused ? 0 : static_cast<int>(total[0]);
  const int wanted = refused ? 0 : static_cast<int>(total[1]);
  const int dropped = refused ? 0 : static_cast<int>(total[2]);
  const int tid = blockIdx.x * kPagesThreads + threadIdx.x;
  const int step = gridDim.x * kPagesThreads;

  auto want_of = [&](int b) {
    return static_cast<int>((static_cast<int64_t>(a.seq[b]) + page_mask) >> a.page_log2);
  };
  // the dropped page of rank k, of row b
  auto dropped_of = [&](int k, int b) {
    return a.tables[b * a.table_stride + want_of(b) + (k - s_drop[b])];
  };
  // the page of wanted rank k; -1 (and the error bit) if the list holds no page there
  auto wanted_page = [&](int k) {
    const int page = k < dropped ? dropped_of(k, row_of(s_drop, a.rows, k))
                                 : a.free_pages[count - 1 - (k - dropped)];
    if (page >= 0 && page < a.num_pages) return page;
    raise_error(a.err, kErrPages);
    return -1;
  };

  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b <= a.rows; b += kPagesThreads) a.cu[b] = refused ? 0 : s_cu[b];
  for (int64_t k0 = static_cast<int64_t>(tid) * kPagesPerThread; k0 < wanted;
       k0 += static_cast<int64_t>(step) * kPagesPerThread) {
    int b = row_of(s_grow, a.rows, static_cast<int>(k0));
#pragma unroll
    for (int i = 0; i < kPagesPerThread; ++i) {
      const int k = static_cast<int>(k0) + i;
      if (k0 + i >= wanted) break;
      while (s_grow[b + 1] <= k) ++b;
      a.tables[b * a.table_stride + a.owned[b] + (k - s_grow[b])] = wanted_page(k);
    }
  }
  for (int64_t k0 = wanted + static_cast<int64_t>(tid) * kPagesPerThread; k0 < dropped;
       k0 += static_cast<int64_t>(step) * kPagesPerThread) {
    int b = row_of(s_drop, a.rows, static_cast<int>(k0));
    int row[kPagesPerThread], page[kPagesPerThread];
#pragma unroll
    for (int i = 0; i < kPagesPerThread; ++i) {
      const int k = static_cast<int>(min(k0 + i, static_cast<int64_t>(dropped) - 1));
      while (s_drop[b + 1] <= k) ++b;
      row[i] = b;
    }
#pragma unroll
    for (int i = 0; i < kPagesPerThread; ++i)
      page[i] = dropped_of(static_cast<int>(min(k0 + i, static_cast<int64_t>(dropped) - 1)), row[i]);
#pragma unroll
    for (int i = 0; i < kPagesPerThread; ++i)
      if (k0 + i < dropped) {
        // (a bad id keeps its place, so that the list's length and order hold;
        // whoever takes it is told again and does not follow it)
        if (page[i] < 0 || page[i] >= a.num_pages) raise_error(a.err, kErrPages);
        a.free_pages[count + dropped - 1 - (k0 + i)] = page[i];
      }
  }

  // slots and positions, kTokensPerThread tokens at a time
  for (int64_t t0 = static_cast<int64_t>(tid) * kTokensPerThread; t0 < a.max_tokens;
       t0 += static_cast<int64_t>(step) * kTokensPerThread) {
    int64_t slot[kTokensPerThread];
    int32_t pos[kTokensPerThread];
    int b = t0 < tokens ? row_of(s_cu, a.rows, static_cast<int>(t0)) : 0;
    int known = -1, page = -1;   // the page index looked up last, and its page
#pragma unroll
    for (int i = 0; i < kTokensPerThread; ++i) {
      const int t = static_cast<int>(t0) + i;
      slot[i] = -1;
      pos[i] = 0;
      if (t0 + i < tokens) {
        while (s_cu[b + 1] <= t) {
          ++b;
          known = -1;
        }
        pos[i] = a.seq[b] - (s_cu[b + 1] - t);
        const int at = pos[i] >> a.page_log2;
        if (at != known) {
          known = at;
          const int owned = a.owned[b];
          if (at < owned) {
            page = a.tables[b * a.table_stride + at];
            if (page < 0 || page >= a.num_pages) {
              raise_error(a.err, kErrPages);
              page = -1;
            }
          } else {
            page = wanted_page(s_grow[b] + (at - owned));
          }
        }
        if (page >= 0)
          slot[i] = (static_cast<int64_t>(page) << a.page_log2) + (pos[i] & page_mask);
      }
    }
    if (t0 + kTokensPerThread <= a.max_tokens) {
      longlong2* s = reinterpret_cast<longlong2*>(a.slots + t0);
      s[0] = make_longlong2(slot[0], slot[1]);
      s[1] = make_longlong2(slot[2], slot[3]);
      *reinterpret_cast<int4*>(a.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
      for (int i = 0; i < kTokensPerThread && t0 + i < a.max_tokens; ++i) {
        a.slots[t0 + i] = slot[i];
        a.positions[t0 + i] = pos[i];
      }
    }
  }

  // commit: by the last CTA, when no other reads the old state any more (the
  // barriers and the counter's acquire and release order their reads before it)
  if (gridDim.x > 1) {
    __syncthreads();
    if (threadIdx.x == 0) {
      uint32_t before;
      asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;"
                   : "=r"(before) : "l"(a.pool + 1) : "memory");
      s_last = before == gridDim.x - 1;
    }
    __syncthreads();
    if (!s_last) return;
    if (threadIdx.x == 0) a.pool[1] = 0;
  } else {
    __syncthreads();
  }
  if (refused) return;
  for (int b = threadIdx.x; b < a.rows; b += kPagesThreads) a.owned[b] = want_of(b);
  if (threadIdx.x == 0) a.pool[0] = count + dropped - wanted;
}

// ---------------------------------------------------------------------------
// Cache write
//
// One thread moves 16 channels (E4M3: two 16-byte loads and one 16-byte store)
// or 8 (bf16) of K and the same of V; the lanes of a (token, head) row are
// neighbours, so loads and stores are whole 128-byte lines in both page
// layouts.  Bound: HBM (3 bytes a value for E4M3, 4 for bf16): 8075 tokens of 16
// heads from a fused QKV projection, 99 MB, 17.1 us from and to cold memory (5.8
// TB/s; 18.1 with 8 resident CTAs an SM that loop), 12.5 us where the buffers
// stay in L2; 64 tokens of 8 heads 2.0 us (launch).
// ---------------------------------------------------------------------------

constexpr int kWriteThreads = 256;

struct WriteArgs {
  const uint16_t* src[2];        // k, v
  uint8_t* dst[2];
  int64_t tok_stride, head_stride;                  // source, elements
  int64_t page_stride, slot_stride, cache_head_stride;   // cache, elements
  const int64_t* slots;
  int64_t num_slots;
  int page_log2, heads;
  uint32_t rows;                 // tokens * heads
  const float* qs;               // E4M3: {qs_q, qs_k, qs_v}
  int32_t* err;
};

__device__ __forceinline__ uint4 ld_stream(const uint16_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// 8 bf16 -> 8 E4M3 codes of fl32(x * qs), the quantisation kernels' cast.
__device__ __forceinline__ uint2 cast8(uint4 x, float qs) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    h[i] = cvt_e4m3x2(__fmul_rn(__uint_as_float(w[i] << 16), qs),
                      __fmul_rn(__uint_as_float(w[i] & 0xFFFF0000u), qs));
  return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

template <bool kFp8>
__global__ void __launch_bounds__(kWriteThreads) kv_write_kernel(const WriteArgs a) {
  constexpr int kLanes = kFp8 ? 8 : 16;             // threads per row
  constexpr int kChannels = kHeadDim / kLanes;
  constexpr int kRowsPerCta = kWriteThreads / kLanes;
  const int c = (threadIdx.x % kLanes) * kChannels;
  const float qs_k = kFp8 ? __ldg(a.qs + 1) : 0.0f, qs_v = kFp8 ? __ldg(a.qs + 2) : 0.0f;
  const uint64_t r = static_cast<uint64_t>(blockIdx.x) * kRowsPerCta + threadIdx.x / kLanes;
  if (r >= a.rows) return;
  const uint32_t t = static_cast<uint32_t>(r) / static_cast<uint32_t>(a.heads);
  const uint32_t h = static_cast<uint32_t>(r) - t * static_cast<uint32_t>(a.heads);
  const int64_t slot = __ldg(reinterpret_cast<const long long*>(a.slots) + t);
  const int64_t from = static_cast<int64_t>(t) * a.tok_stride + h * a.head_stride + c;
  const uint16_t* k = a.src[0] + from;
  const uint16_t* v = a.src[1] + from;
  // the loads do not wait for the slot
  const uint4 k0 = ld_stream(k), v0 = ld_stream(v);
  uint4 k1 = make_uint4(0, 0, 0, 0), v1 = k1;
  if (kFp8) {
    k1 = ld_stream(k + 8);
    v1 = ld_stream(v + 8);
  }
  if (slot < 0) return;
  if (slot >= a.num_slots) {
    raise_error(a.err, kErrPages);
    return;
  }
  const int64_t to = (slot >> a.page_log2) * a.page_stride +
                     (slot & ((1 << a.page_log2) - 1)) * a.slot_stride +
                     h * a.cache_head_stride + c;
  if (kFp8) {
    const uint2 ka = cast8(k0, qs_k), kb = cast8(k1, qs_k);
    const uint2 va = cast8(v0, qs_v), vb = cast8(v1, qs_v);
    *reinterpret_cast<uint4*>(a.dst[0] + to) = make_uint4(ka.x, ka.y, kb.x, kb.y);
    *reinterpret_cast<uint4*>(a.dst[1] + to) = make_uint4(va.x, va.y, vb.x, vb.y);
  } else {
    *reinterpret_cast<uint4*>(a.dst[0] + 2 * to) = k0;
    *reinterpret_cast<uint4*>(a.dst[1] + 2 * to) = v0;
  }
}

// ---------------------------------------------------------------------------
// Accepted path -> tail
//
// Row b's accepted nodes path[0] < path[1] < ... move to nodes 0, 1, ...: node
// i's new place never lies behind its old one nor behind a later node's, so a
// thread that reads a batch of its 16-byte column before it writes that batch
// moves in place, with no other thread involved.  Bound: latency (path, table
// and row are dependent loads), so the batches keep eight rows in flight: 4
// trees of 25 nodes 3.3 us, 96 trees of 64 nodes 4.1 us.
// ---------------------------------------------------------------------------

constexpr int kKeepThreads = 128;
constexpr int kKeepBatch = 8;

struct KeepArgs {
  uint8_t* cache[2];
  int64_t page_stride, slot_stride, head_stride;   // bytes
  int num_pages, page_log2;
  const int32_t* tables;
  int64_t table_stride;
  int width;
  const int32_t* seq;
  const int32_t* cu;
  const int32_t* paths;
  int64_t path_stride;
  int depth;
  const int32_t* keep;
  int heads, vecs_log2;            // 16-byte vectors of a head row
  int32_t* err;
};

__global__ void __launch_bounds__(kKeepThreads) kv_keep_kernel(const KeepArgs a) {
  const int b = blockIdx.x;
  const int32_t* path = a.paths + b * a.path_stride;
  const int keep = a.keep[b], n = a.cu[b + 1] - a.cu[b], seq = a.seq[b];
  bool bad = keep < 0 || keep > a.depth || keep > n || n < 0 || n > seq ||
             seq > (static_cast<int64_t>(a.width) << a.page_log2);
  if (!bad)
    for (int i = threadIdx.x; i < keep; i += kKeepThreads)
      if (path[i] < 0 || path[i] >= n || (i > 0 && path[i] <= path[i - 1])) bad = true;
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0 && blockIdx.y == 0) raise_error(a.err, kErrSeqlens);
    return;
  }
  // this thread's 16-byte column: (K or V, head, vector)
  const int col = blockIdx.y * kKeepThreads + threadIdx.x;
  const int vec = col & ((1 << a.vecs_log2) - 1);
  const int hk = col >> a.vecs_log2;
  if (hk >= 2 * a.heads) return;
  const int which = hk >= a.heads;
  uint8_t* base = a.cache[which] + (hk - which * a.heads) * a.head_stride + vec * 16;
  const int32_t* table = a.tables + b * a.table_stride;
  const int ctx = seq - n, page_mask = (1 << a.page_log2) - 1;
  auto row = [&](int node) -> uint4* {
    const int pos = ctx + node;
    const int page = table[pos >> a.page_log2];
    if (page < 0 || page >= a.num_pages) return nullptr;
    return reinterpret_cast<uint4*>(base + page * a.page_stride +
                                    (pos & page_mask) * a.slot_stride);
  };
  bool lost = false;
  for (int i0 = 0; i0 < keep; i0 += kKeepBatch) {
    uint4 x[kKeepBatch];
    uint4* to[kKeepBatch];
#pragma unroll
    for (int u = 0; u < kKeepBatch; ++u) {
      to[u] = nullptr;
      const int i = i0 + u;
      if (i < keep && path[i] != i) {
        const uint4* from = row(path[i]);
        uint4* dst = row(i);
        lost |= !from || !dst;
        if (from && dst) {
          x[u] = *from;
          to[u] = dst;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kKeepBatch; ++u)
      if (to[u]) *to[u] = x[u];
  }
  if (lost) raise_error(a.err, kErrPages);
}

}  // namespace

cudaError_t launch_assign_pages(const AssignPagesLaunch& p, cudaStream_t stream) {
  PagesArgs a;
  a.seq = p.seq;
  a.fresh = p.fresh;
  a.tables = p.tables;
  a.table_stride = p.table_stride;
  a.width = p.width;
  a.owned = p.owned;
  a.free_pages = p.free_pages;
  a.num_pages = p.num_pages;
  a.pool = p.pool;
  a.rows = p.rows;
  a.page_log2 = p.page_log2;
  a.max_tokens = p.max_tokens;
  a.cu = p.cu;
  a.slots = p.slots;
  a.positions = p.positions;
  a.err = p.err;
  // enough CTAs for the tokens, and for the pages that rows may take or give
  // back (the pool's or the tables', whichever is fewer: two rounds of a CTA)
  const int64_t by_tokens =
      (static_cast<int64_t>(p.max_tokens) + kPagesThreads * kTokensPerThread - 1) /
      (kPagesThreads * kTokensPerThread);
  const int64_t held = static_cast<int64_t>(p.rows) * p.width;
  const int64_t by_pages =
      (held < p.num_pages ? held : p.num_pages) / (2 * kPagesThreads * kPagesPerThread);
  int64_t grid = by_tokens > by_pages ? by_tokens : by_pages;
  if (grid < 1) grid = 1;
  if (grid > 148) grid = 148;
  const size_t smem = 3 * (static_cast<size_t>(p.rows) + 1) * sizeof(int32_t);
  // a launch gets 48 KB unasked, for these sums and the kernel's own 400 bytes
  // of shared variables (1024 are more than enough)
  if (smem + 1024 > 48 * 1024) {
    // (always the largest size: calls of other threads with more rows rely on it)
    constexpr int kMost = 3 * (kMaxPageRows + 1) * static_cast<int>(sizeof(int32_t));
    static_assert(kMost <= 227 * 1024 - 1024, "shared memory of a CTA");
    cudaError_t e = cudaFuncSetAttribute(assign_pages_kernel,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
    if (e != cudaSuccess) return e;
  }
  assign_pages_kernel<<<static_cast<unsigned>(grid), kPagesThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_kv_write(const KvWriteLaunch& p, cudaStream_t stream) {
  WriteArgs a;
  a.src[0] = static_cast<const uint16_t*>(p.k);
  a.src[1] = static_cast<const uint16_t*>(p.v);
  a.dst[0] = static_cast<uint8_t*>(p.cache.k);
  a.dst[1] = static_cast<uint8_t*>(p.cache.v);
  a.tok_stride = p.tok_stride;
  a.head_stride = p.head_stride;
  a.page_stride = p.cache.page_stride;
  a.slot_stride = p.cache.slot_stride;
  a.cache_head_stride = p.cache.head_stride;
  a.slots = p.slots;
  a.num_slots = static_cast<int64_t>(p.cache.num_pages) << p.cache.page_log2;
  a.page_log2 = p.cache.page_log2;
  a.heads = p.cache.heads;
  a.rows = static_cast<uint32_t>(p.tokens * p.cache.heads);
  a.qs = p.qs;
  a.err = p.err;
  const int rows_per_cta = kWriteThreads / (p.cache.fp8 ? 8 : 16);
  const int64_t grid = (static_cast<int64_t>(a.rows) + rows_per_cta - 1) / rows_per_cta;
  if (p.cache.fp8)
    kv_write_kernel<true><<<static_cast<unsigned>(grid), kWriteThreads, 0, stream>>>(a);
  else
    kv_write_kernel<false><<<static_cast<unsigned>(grid), kWriteThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_kv_keep(const KvKeepLaunch& p, cudaStream_t stream) {
  const int esz = p.cache.fp8 ? 1 : 2;
  KeepArgs a;
  a.cache[0] = static_cast<uint8_t*>(p.cache.k);
  a.cache[1] = static_cast<uint8_t*>(p.cache.v);
  a.page_stride = p.cache.page_stride * esz;
  a.slot_stride = p.cache.slot_stride * esz;
  a.head_stride = p.cache.head_stride * esz;
  a.num_pages = p.cache.num_pages;
  a.page_log2 = p.cache.page_log2;
  a.tables = p.tables;
  a.table_stride = p.table_stride;
  a.width = p.width;
  a.seq = p.seq;
  a.cu = p.cu;
  a.paths = p.paths;
  a.path_stride = p.path_stride;
  a.depth = p.depth;
  a.keep = p.keep;
  a.heads = p.cache.heads;
  a.vecs_log2 = p.cache.fp8 ? 3 : 4;
  a.err = p.err;
  const int64_t cols = static_cast<int64_t>(2 * a.heads) << a.vecs_log2;
  const dim3 grid(static_cast<unsigned>(p.rows),
                  static_cast<unsigned>((cols + kKeepThreads - 1) / kKeepThreads));
  kv_keep_kernel<<<grid, kKeepThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace fp8attn
