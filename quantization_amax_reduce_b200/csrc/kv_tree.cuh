// Device code shared by the two attention kernels over the paged KV cache
// (kv_tree.cu): arguments, the work list, the TMA producers and the warps that
// prepare Q and V.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.h"
#include "sm100_ptx.cuh"
#include "state.cuh"

namespace fp8attn {

namespace kv_tree {

constexpr int kTile = 128;                 // keys of a tile
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kPOffset = 8.0f;           // log2 of P at the reference
constexpr float kRefLag = 7.0f;
constexpr int kMaxCtas = 148;              // one per SM
// What a unit costs beside its tiles (its Q, the way through the pipeline, its
// epilogue), in tiles: ranges are cut by tiles plus this, or a CTA whose
// requests are short works through a dozen units while others read one long
// one.  128 chains of 4 over 5 to 300 tokens: 73 us at 0, 60 at 2, 58 at 4, 63
// at 10; 16 trees of up to 25 over 100 to 5000 tokens (bf16): 81, 56, 49, 53.
constexpr int kUnitCost = 4;
constexpr int kPrepWarps = 4, kPrepThreads = 32 * kPrepWarps;

struct TreeArgs {
  const uint16_t* q;
  int64_t q_tok_stride, q_head_stride;
  const uint8_t* v;                      // V cache, for the non-finite rows
  int64_t page_stride, slot_stride, head_stride;   // elements
  int num_pages, page_log2, kv_heads, group;
  uint32_t group_magic;                  // ceil(2^32 / group), 0 for a group of one
  const int32_t* tables;
  int64_t table_stride;
  int width;
  const int32_t* seq;
  const int32_t* cu;
  int rows, max_q, max_seqlen, total_q;
  const float* descale;
  const unsigned long long* mask;
  int mask_words;
  float softmax_scale;
  __nv_bfloat16* out;
  float* part_o;                         // [2 CTAs][R][128]
  float2* part_ml;                       // [2 CTAs][R] {ref, sum}
  struct JoinInfo* join;                 // [CTAs] the unit that begins in a CTA and leaves it
  int32_t* err;
  int stall_k, stall_v;                  // tile of a CTA at which its producer stops (self-test)
};

// A CTA's tiles [t0, t1) of one unit.
struct Segment {
  int b, head, rt;       // request, KV head, row tile
  int seq, q0, n;
  int tiles, t0, t1;     // tiles of the unit; this CTA's (none: the end)
};

// A unit of several pieces: they lie in this CTA and the next ones (none: no
// such unit).
struct JoinInfo {
  int q0, n, head, rt, pieces;
};

// What a unit's rows stand for.  Units u and u + 1 may be in use while unit
// u + 2's slot is written.
template <int R>
struct UnitRows {
  alignas(16) float factor[R];           // score -> log2 units
  int one_factor;                        // they are all the same (up to 32 rows)
  int out_row[R];                        // row of `out`, -1 = none
  int node[R];                           // -1 = none
  Segment seg;
};

__device__ __forceinline__ void raise_error(int32_t* err, uint32_t bits) {
  if (err) atomicOr(reinterpret_cast<unsigned int*>(err), bits);
}

__device__ __forceinline__ void group_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Does any of the group's threads say yes?
__device__ __forceinline__ bool group_any(int id, int threads, bool yes) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 q, %1, 0;\n\t"
      "bar.red.or.pred p, %2, %3, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(yes)), "r"(id), "r"(threads)
      : "memory");
  return r != 0;
}

template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[N]) {
  if constexpr (N == 8) tmem_ld8(taddr, r);
  else tmem_ld16(taddr, r);
}

template <int N>
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&r)[N]) {
  if constexpr (N == 8) tmem_st8(taddr, r);
  else tmem_st16(taddr, r);
}

// A pair times a power of two (exact but for what leaves the type's range).
__device__ __forceinline__ uint32_t scale_f16x2(uint32_t x, float s) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&x));
  return cvt_f16x2(f.x * s, f.y * s);
}

__device__ __forceinline__ uint32_t scale_bf16x2(uint32_t x, float s) {
  return cvt_bf16x2(__uint_as_float(x << 16) * s, __uint_as_float(x & 0xFFFF0000u) * s);
}

// Reduces N columns (8 or 16) over the warp's lanes: lane l
// gets column l % N.  N - 1 + log2(32 / N) shuffles instead of 5 N.
template <int N, bool kMax>
__device__ __forceinline__ float reduce_columns(float (&v)[N], int lane) {
  auto join = [](float a, float b) { return kMax ? fmaxf(a, b) : a + b; };
#pragma unroll
  for (int off = N / 2; off >= 1; off /= 2) {
    const bool up = (lane & off) != 0;
#pragma unroll
    for (int i = 0; i < off; ++i) {
      const float send = up ? v[i] : v[i + off];
      const float mine = up ? v[i + off] : v[i];
      v[i] = join(mine, __shfl_xor_sync(0xffffffffu, send, off));
    }
  }
#pragma unroll
  for (int off = N; off < 32; off *= 2)
    v[0] = join(v[0], __shfl_xor_sync(0xffffffffu, v[0], off));
  return v[0];
}

// Transposes a 32 x 32 bit matrix held one row per lane.
__device__ __forceinline__ uint32_t transpose_bits(uint32_t x, int lane) {
  uint32_t m = 0x0000FFFFu;
#pragma unroll
  for (int j = 16; j >= 1; j >>= 1, m ^= m << j) {
    const uint32_t y = __shfl_xor_sync(0xffffffffu, x, j);
    x = (lane & j) ? (x & ~m) | ((y >> j) & m) : (x & m) | ((y & m) << j);
  }
  return x;
}

// Bits [j0, j0 + 32) of a mask row of `words` words; j0 > -32.
__device__ __forceinline__ uint32_t mask_bits(const unsigned long long* row, int words, int j0) {
  if (j0 < 0) return static_cast<uint32_t>(__ldg(row) << -j0);
  const int w = j0 >> 6, sh = j0 & 63;
  if (w >= words) return 0;
  uint64_t v = __ldg(row + w) >> sh;
  if (sh > 32 && w + 1 < words) v |= __ldg(row + w + 1) << (64 - sh);
  return static_cast<uint32_t>(v);
}

__device__ __forceinline__ uint32_t low_bits(int n) {   // the n lowest bits, 0 <= n
  return n >= 32 ? 0xffffffffu : (1u << n) - 1;
}

// ---------------------------------------------------------------------------
// Work list: the units in order (request, head, row tile), each kUnitCost items
// and then an item per tile, cut into a range of items per CTA.  Every role
// walks the same segments (a CTA's tiles of one unit).
// ---------------------------------------------------------------------------

// Node of a query row: row / group, exact while row * group < 2^32.
__device__ __forceinline__ int node_of(const TreeArgs& a, int row) {
  return a.group_magic ? static_cast<int>(__umulhi(static_cast<uint32_t>(row), a.group_magic)) : row;
}

struct Request {
  int seq, q0, n, tiles, row_tiles;
  int span;              // items of a unit: its cost and its tiles
  __device__ __forceinline__ int work(int kv_heads) const { return kv_heads * row_tiles * span; }
};

// A request's lengths; false if they are inconsistent (it then has no work).
template <int R>
__device__ __forceinline__ bool read_request(const TreeArgs& a, int b, Request& r) {
  r.seq = a.seq[b];
  r.q0 = a.cu[b];
  const int q1 = a.cu[b + 1];
  r.n = q1 - r.q0;
  const bool ok = r.q0 >= 0 && q1 >= r.q0 && q1 <= a.total_q && r.n <= a.max_q && r.seq >= r.n &&
                  r.seq <= a.max_seqlen &&
                  r.seq <= static_cast<int64_t>(a.width) << a.page_log2 &&
                  (!a.mask || r.n <= 64ll * a.mask_words);
  r.tiles = ok ? (r.seq + kTile - 1) / kTile : 0;
  r.row_tiles = ok ? (r.n * a.group + R - 1) / R : 0;
  r.span = kUnitCost + r.tiles;
  return ok;
}

// chunk[i] = items of the requests before thread i's; chunk[kThreads] = all.
// Returns whether this thread met an inconsistent request.
template <int R, int kThreads>
__device__ bool scan_requests(const TreeArgs& a, int* chunk, int* warp_sums) {
  const int per = (a.rows + kThreads - 1) / kThreads;
  const int first = min(a.rows, static_cast<int>(threadIdx.x) * per);
  const int last = min(a.rows, first + per);
  bool bad = false;
  int sum = 0;
  for (int b = first; b < last; ++b) {
    Request r;
    bad |= !read_request<R>(a, b, r);
    sum += r.work(a.kv_heads);
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = sum;
#pragma unroll
  for (int off = 1; off < 32; off *= 2) {
    const int up = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += up;
  }
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  int at = incl - sum;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const int s = warp_sums[w];
    at += w < warp ? s : 0;
  }
  chunk[threadIdx.x] = at;
  if (threadIdx.x == kThreads - 1) chunk[kThreads] = at + sum;
  return bad;   // (the caller syncs)
}

// The request that a work item belongs to.
template <int R, int kThreads>
struct Finder {
  Request r;
  int b = -1, start = 0, stop = 0;   // request, its first item, end of its chunk
  // (the whole warp)
  __device__ __forceinline__ void seek(const TreeArgs& a, const int* chunk, int w) {
    if (b >= 0 && w < start + r.work(a.kv_heads)) return;
    while (b >= 0 && b + 1 < stop) {   // a neighbour of the same chunk
      start += r.work(a.kv_heads);
      read_request<R>(a, ++b, r);
      if (w < start + r.work(a.kv_heads)) return;
    }
    // the last chunk that starts at or before w: 32 lanes probe every kStep-th,
    // then the ones after the last that does
    constexpr int kStep = (kThreads + 31) / 32;
    const int lane = threadIdx.x & 31;
    int lo = lane * kStep;
    lo = kStep * (__popc(__ballot_sync(0xffffffffu, lo < kThreads && chunk[min(lo, kThreads)] <= w)) - 1);
    const int probe = lo + lane;
    lo += __popc(__ballot_sync(0xffffffffu, lane < kStep && probe < kThreads &&
                                                chunk[min(probe, kThreads)] <= w)) - 1;
    const int per = (a.rows + kThreads - 1) / kThreads;
    b = lo * per;
    stop = min(a.rows, b + per);
    start = chunk[lo];
    read_request<R>(a, b, r);
    while (w >= start + r.work(a.kv_heads)) {
      start += r.work(a.kv_heads);
      read_request<R>(a, ++b, r);
    }
  }
};

// The pieces of a unit that begins with `s`, which its CTA does not finish.
__device__ __forceinline__ JoinInfo join_info(const Segment& s, int per) {
  return {s.q0, s.n, s.head, s.rt, 1 + (s.tiles - s.t1 + per - 1) / per};
}

template <int R, int kThreads>
struct Walker {
  Finder<R, kThreads> find;
  int w, end;
  int head = 0, rt = -1;     // the unit handed out last (its last tile was, too)
  __device__ __forceinline__ void init(const int* chunk, int ctas) {
    const int total = chunk[kThreads];
    const int per = tree_items_per_cta(total, ctas);
    const int64_t from = static_cast<int64_t>(blockIdx.x) * per;
    w = static_cast<int>(min(from, static_cast<int64_t>(total)));
    end = static_cast<int>(min(from + per, static_cast<int64_t>(total)));
  }
  // (the whole warp)
  __device__ __forceinline__ bool next(const TreeArgs& a, const int* chunk, Segment& s) {
    if (w >= end) return false;
    const bool first = rt < 0;
    const int old = find.b;
    find.seek(a, chunk, w);
    const Request& r = find.r;
    int x0 = 0;
    if (first) {             // somewhere inside a unit
      const int local = w - find.start;
      const int unit = local / r.span;
      head = unit / r.row_tiles;
      rt = unit - head * r.row_tiles;
      x0 = local - unit * r.span;
    } else if (find.b != old) {
      head = rt = 0;
    } else if (++rt == r.row_tiles) {
      rt = 0;
      ++head;
    }
    s.b = find.b;
    s.seq = r.seq;
    s.q0 = r.q0;
    s.n = r.n;
    s.tiles = r.tiles;
    s.head = head;
    s.rt = rt;
    const int x1 = min(r.span, x0 + (end - w));
    w += x1 - x0;
    s.t0 = max(0, x0 - kUnitCost);
    s.t1 = max(0, x1 - kUnitCost);
    return s.t1 > 0;         // (none: the range ends before the unit's first tile)
  }
};

// ---------------------------------------------------------------------------
// Waits.  One that gives up sets the abort flag, which ends all other waits at
// once.  Warps that share a barrier must still agree on what comes next: the
// preparing warps go through all of their units, but hand out no more of them,
// and the softmax warps run on without data to the end of their unit, where
// they vote on whether there is a next one.  Nothing is written out then.  The
// flag may rise between two lanes' looks at it, so what a warp does as one goes
// by its vote (any_aborted).  (The whole warp tests a barrier: 64 cycles when
// the phase is over already, against 117 for one lane and a warp sync.)
// ---------------------------------------------------------------------------

struct Waits {
  int* abort_flag;       // shared memory
  int32_t* err;
  int lane;
  __device__ __forceinline__ bool aborted() const {
    return *const_cast<volatile int*>(abort_flag) != 0;
  }
  // the same for all lanes
  __device__ __forceinline__ bool any_aborted() const {
    return __any_sync(0xffffffffu, aborted());
  }
  __device__ __forceinline__ void wait(uint64_t* bar, uint32_t parity) const {
    if (!mbar_wait(bar, parity, const_cast<volatile int*>(abort_flag))) {
      if (!aborted()) raise_error(err, kErrTimeout);
      *const_cast<volatile int*>(abort_flag) = 1;
    }
    __syncwarp();
  }
  // one arrival for the warp
  __device__ __forceinline__ void arrive(uint64_t* bar) const {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  }
};

// ---------------------------------------------------------------------------
// TMA producer of K or of V (a warp each: neither waits for the other's
// stages): a box per page, one lane per page, page ids looked up a tile ahead.
// A page id outside the cache is outside the tensor map: zeros arrive.  Before
// stage i's n-th refill (n >= 1) it waits for phase n - 1 of free1[i], and of
// free2[i] if there is one.  After an abort there are no more copies: a stage
// may then be given back whose last one never landed, and its barrier takes
// another's bytes only in the next phase.
// ---------------------------------------------------------------------------

template <int R, int kThreads, bool kFp8>
__device__ __forceinline__ void produce(const TreeArgs& a, const Waits& w, const int* chunk, const CUtensorMap* map,
                        bool is_k, uint8_t* ring, int stages, uint64_t* full, uint64_t* free1,
                        uint64_t* free2) {
  constexpr int kBytes = kFp8 ? 16384 : 32768;   // of a tile
  const int page = 1 << a.page_log2;
  const int box = min(page, kTile);
  const int box_log2 = min(a.page_log2, 7);
  Walker<R, kThreads> walk;
  walk.init(chunk, gridDim.x);
  Segment seg;
  int g = 0, stage = 0, turn = 0;
  const int stall = is_k ? a.stall_k : a.stall_v;
  bool stop = false;
  while (!stop && walk.next(a, chunk, seg)) {
    const int32_t* table = a.tables + seg.b * a.table_stride;
    // this lane's first key of a tile; it has a page to load if that lies before
    // `last`
    const int last = w.lane < kTile >> box_log2 ? seg.seq : 0;
    auto first_key = [&](int t) { return t * kTile + (w.lane << box_log2); };
    auto look_up = [&](int t) {
      if (first_key(t) >= last) return 0;
      return __ldg(table + (first_key(t) >> a.page_log2));
    };
    int next_id = look_up(seg.t0);
    for (int t = seg.t0; t < seg.t1; ++t, ++g) {
      const int id = next_id;
      if (t + 1 < seg.t1) next_id = look_up(t + 1);
      const bool load = first_key(t) < last;   // (whatever its id: no id means "none")
      if (is_k && load && (id < 0 || id >= a.num_pages)) raise_error(a.err, kErrPages);
      const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, load)) * box * (kFp8 ? 128 : 256);
      const int row = a.page_log2 > 7 ? (t * kTile) & (page - 1) : 0;
      if (turn > 0) {
        w.wait(&free1[stage], (turn - 1) & 1);
        if (free2) w.wait(&free2[stage], (turn - 1) & 1);
      }
      stop = w.any_aborted() || g == stall;
      if (stop) break;
      if (w.lane == 0) mbar_expect_tx(&full[stage], bytes);
      __syncwarp();
      if (load) {
        uint8_t* dst = ring + stage * kBytes + w.lane * box * 128;
        tma_load_4d(dst, map, &full[stage], 0, seg.head, row, id);
        if (!kFp8) tma_load_4d(dst + 16384, map, &full[stage], 64, seg.head, row, id);
      }
      __syncwarp();
      if (++stage == stages) stage = 0, ++turn;
    }
  }
  // no copy may still be landing when the CTA leaves
  if (w.lane == 0)
    for (int i = max(0, g - stages); i < g; ++i)
      mbar_wait(&full[i % stages], (i / stages) & 1, nullptr);
  __syncwarp();
}

// 128-row tiles with at most 64 rows hold them twice: rows 64 to 127 are rows 0
// to 63 again, and take the second half of a tile's keys.
template <int R>
__device__ __forceinline__ bool is_doubled(const TreeArgs& a, const Segment& s) {
  return R == 128 && s.n * a.group - s.rt * R <= 64;
}

// ---------------------------------------------------------------------------
// Q of a unit: a half warp per row, 8 channels a lane, four rows of a half warp
// at a time, the first four loaded a unit ahead.  K-major rows of 128 bytes,
// 128-byte swizzle; bf16: two 64-channel halves; E4M3: hi tile, then the
// remainders (times kLoScale) R rows on.
// ---------------------------------------------------------------------------

template <int R>
struct QLoads {
  static constexpr int kRows = kPrepThreads / 16;           // rows of one load
  static constexpr int kAll = R / kRows, kLoads = kAll < 4 ? kAll : 4;
  uint4 x[kLoads];
  __device__ __forceinline__ void load(const TreeArgs& a, const Segment& s, int tid, int first) {
    const int same = is_doubled<R>(a, s) ? 63 : R - 1;
#pragma unroll
    for (int it = 0; it < kLoads; ++it) {
      const int row = s.rt * R + (((first + it) * kRows + (tid >> 4)) & same);
      const int node = node_of(a, row), gq = row - node * a.group;
      x[it] = make_uint4(0, 0, 0, 0);
      if (node < s.n)
        x[it] = __ldg(reinterpret_cast<const uint4*>(a.q + (s.q0 + node) * a.q_tok_stride +
                                                     (s.head * a.group + gq) * a.q_head_stride +
                                                     (tid & 15) * 8));
    }
  }
};

// 2^e <= amax < 2^(e + 1) for bf16 bits; 2^(7 - e) and 2^(e - 7) are normal.
__device__ __forceinline__ int exponent_of(uint32_t bits) {
  return max(static_cast<int>(bits >> 7) - 127, -119);
}

__device__ __forceinline__ float power_of_two(int e) {
  return __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
}

// |x| max of a row's 128 channels, as bf16 bits.
__device__ __forceinline__ uint32_t row_amax(uint4 x) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
  m = max(m & 0xFFFFu, m >> 16);
#pragma unroll
  for (int off = 8; off >= 1; off /= 2) m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
  return m;
}

// 8 channels of row r, scaled by 2^(7 - e), as two E4M3 numbers each.
template <int R, int kLoScale>
__device__ __forceinline__ void split_q(uint4 x, int e, bool whole, uint8_t* sq, int r, int c) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  const float up = power_of_two(7 - e);
  uint32_t hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float x0 = __uint_as_float(w[i] << 16) * up;
    const float x1 = __uint_as_float(w[i] & 0xFFFF0000u) * up;
    const uint32_t h = cvt_e4m3x2(x0, x1);
    const uint32_t hf = cvt_f16x2_from_e4m3x2(h);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hf));
    const uint32_t l = cvt_e4m3x2((x0 - f.x) * kLoScale, (x1 - f.y) * kLoScale);
    hi[i >> 1] |= (whole ? h : 0x7F7Fu) << (16 * (i & 1));
    lo[i >> 1] |= (whole ? l : 0x7F7Fu) << (16 * (i & 1));
  }
  uint8_t* to = sq + (r >> 3) * 1024 + (r & 7) * 128 + (((c >> 1) ^ (r & 7)) << 4) + (c & 1) * 8;
  *reinterpret_cast<uint2*>(to) = make_uint2(hi[0], hi[1]);
  *reinterpret_cast<uint2*>(to + R * 128) = make_uint2(lo[0], lo[1]);
}

template <int R, bool kFp8, int kLoScale>
__device__ __forceinline__ void store_q(const TreeArgs& a, const Segment& s, QLoads<R>& q,
                                        uint8_t* sq, UnitRows<R>& rows, uint2* row_max,
                                        int barrier, float unit_factor, int tid, bool hand_out) {
  constexpr int kLoads = QLoads<R>::kLoads, kRows = QLoads<R>::kRows, kAll = QLoads<R>::kAll;
  const int c = tid & 15, lane = tid & 31;
  // a row with Inf or NaN becomes NaN throughout (E4M3)
  if constexpr (kFp8 && kAll == kLoads) {
    uint32_t amax[kLoads], most = 0, least = 0xffffffffu;
#pragma unroll
    for (int it = 0; it < kLoads; ++it) {
      const uint32_t m = row_amax(q.x[it]);
      amax[it] = m;
      if (m < 0x7F80u) most = max(most, m);
      if (m != 0) least = min(least, m);
    }
    most = __reduce_max_sync(0xffffffffu, most);
    least = __reduce_min_sync(0xffffffffu, least);
    if (lane == 0) row_max[tid >> 5] = make_uint2(most, least);
    group_sync(barrier, kPrepThreads);
#pragma unroll
    for (int i = 0; i < kPrepWarps; ++i) {
      const uint2 m = row_max[i];
      most = max(most, m.x);
      least = min(least, m.y);
    }
    // rows within 2^4 of the largest share its scale: a factor in a register
    // instead of one in shared memory per column; otherwise each has its own
    const bool shared = most <= (least & 0x7F80u) + (4u << 7) + 127u;
    if (tid == 0) rows.one_factor = shared;
#pragma unroll
    for (int it = 0; it < kLoads; ++it) {
      const int r = it * kRows + (tid >> 4);
      const int e = exponent_of(shared ? most : amax[it]);
      split_q<R, kLoScale>(q.x[it], e, amax[it] < 0x7F80u, sq, r, c);
      if (c == 0) rows.factor[r] = unit_factor * power_of_two(e - 7);
    }
  } else {
    // (rolled, the next rows on their way while these are stored)
#pragma unroll 1
    for (int first = 0; first < kAll; first += kLoads) {
      QLoads<R> now = q;
      if (first + kLoads < kAll) q.load(a, s, tid, first + kLoads);
#pragma unroll
      for (int it = 0; it < kLoads; ++it) {
        const int r = (first + it) * kRows + (tid >> 4);
        if constexpr (kFp8) {
          const uint32_t m = row_amax(now.x[it]);
          const int e = exponent_of(m);
          split_q<R, kLoScale>(now.x[it], e, m < 0x7F80u, sq, r, c);
          if (c == 0) rows.factor[r] = unit_factor * power_of_two(e - 7);
        } else {
          *reinterpret_cast<uint4*>(sq + (c >> 3) * (R * 128) + (r >> 3) * 1024 + (r & 7) * 128 +
                                    (((c & 7) ^ (r & 7)) << 4)) = now.x[it];
        }
      }
    }
    if (!kFp8 && tid < R) rows.factor[tid] = unit_factor;
    if (!kFp8 && tid == 0) rows.one_factor = 1;
  }
  if (tid < R && hand_out) {
    const int row = s.rt * R + (is_doubled<R>(a, s) ? tid & 63 : tid);
    const int node = node_of(a, row), gq = row - node * a.group;
    const bool live = node < s.n;
    rows.node[tid] = live ? node : -1;
    rows.out_row[tid] = live ? (s.q0 + node) * (a.kv_heads * a.group) + s.head * a.group + gq : -1;
  }
  if (tid == 0 && hand_out) rows.seg = s;
  fence_proxy_async();
}

// ---------------------------------------------------------------------------
// V of a tile.  In tiles that hold nodes, rows past the sequence, up to the 16
// that a product takes at a time, become zeros, and so do the non-finite
// elements of nodes, which a query that does not see
// the node must not meet as 0 x Inf: the epilogue adds them.  Both return
// whether this thread met such an element; pos0 = position of the tile's first
// key, nodes begin at position ctx.
// ---------------------------------------------------------------------------

// E4M3 -> f16 into two 64-channel halves of 128-byte rows, 128-byte swizzle.
// A thread's pieces of 16 channels: for i = 0..7, piece 4 h + (lane & 3), h =
// i & 1, of a row of the eight from 32 warp + 8 (i / 2) on.  It becomes pieces
// 2 (lane & 3) and + 1 of half h.  Of the eight lanes that share a bank cycle
// four have row p and four row p ^ 5: bit 2 apart their reads, bit 0 apart
// their writes fall into different banks.  `ready` runs before the destination
// is written, `taken` when the source may be overwritten: behind the proxy
// fence, since TMA will (an arrival right behind the loads was seen to overtake
// the last of them).
template <int kBatch, class Taken, class Ready>
__device__ __forceinline__ bool widen_v(const uint8_t* src, uint8_t* wide, int tid, bool tail,
                                        int pos0, int ctx, int seq, Taken taken, Ready ready) {
  bool wild = false;
  const int c = tid & 3, p = (tid >> 3) & 3, r = (tid & 4) ? p ^ 5 : p;
  const int row = (tid >> 5) * 32 + r;               // and 8 (i / 2) on
  const uint8_t* from = src + row * 128;
  const int f0 = (c ^ r) << 4, f1 = ((c + 4) ^ r) << 4;
  uint8_t* to = wide + row * 128;
  const int t0 = ((2 * c) ^ r) << 4, t1 = ((2 * c + 1) ^ r) << 4;
#pragma unroll 1
  for (int i0 = 0; i0 < 8; i0 += kBatch) {
    uint4 x[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      x[i] = *reinterpret_cast<const uint4*>(from + (i0 + i) / 2 * 1024 + (i & 1 ? f1 : f0));
    if (tail) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int pos = pos0 + row + (i0 + i) / 2 * 8;
        uint32_t* w = &x[i].x;
        uint32_t nan = 0;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const uint32_t m = pos >= seq   ? 0xffffffffu
                             : pos >= ctx ? __vcmpeq4(w[u] & 0x7F7F7F7Fu, 0x7F7F7F7Fu)
                                          : 0u;
          w[u] &= ~m;
          nan |= m;
        }
        wild |= nan != 0 && pos < seq;
      }
    }
    if (i0 == 0) ready();
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      uint32_t f[8];
#pragma unroll
      for (int u = 0; u < 4; ++u) cvt_f16x4_from_e4m3x4((&x[i].x)[u], f[2 * u], f[2 * u + 1]);
      uint8_t* d = to + (i & 1) * 16384 + (i0 + i) / 2 * 1024;
      *reinterpret_cast<uint4*>(d + t0) = make_uint4(f[0], f[1], f[2], f[3]);
      *reinterpret_cast<uint4*>(d + t1) = make_uint4(f[4], f[5], f[6], f[7]);
    }
  }
  fence_proxy_async();
  taken();
  return wild;
}

// A bf16 tile that holds nodes, in place: 16 lanes a row.
__device__ __forceinline__ bool mend_v(uint8_t* src, int tid, int pos0, int ctx, int seq) {
  bool wild = false;
  const int last = min(kTile, (seq - pos0 + 15) & ~15);
  uint8_t* piece = src + ((tid >> 3) & 1) * 16384 + (tid & 7) * 16;
  for (int row = max(0, ctx - pos0) + (tid >> 4); row < last; row += kPrepThreads / 16) {
    uint4* p = reinterpret_cast<uint4*>(piece + row * 128);
    if (pos0 + row >= seq) {
      *p = make_uint4(0, 0, 0, 0);
      continue;
    }
    uint4 x = *p;
    uint32_t* w = &x.x;
    uint32_t found = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t m = __vcmpeq2(w[u] & 0x7F807F80u, 0x7F807F80u);
      w[u] &= ~m;
      found |= m;
    }
    if (found) *p = x;
    wild |= found != 0;
  }
  fence_proxy_async();
  return wild;
}

// A non-finite element of the V cache as fp32, 0 for a finite one.
template <bool kFp8>
__device__ __forceinline__ float wild_value(const uint8_t* v, int64_t at) {
  if (kFp8) return (v[at] & 0x7Fu) == 0x7Fu ? __uint_as_float(0x7FC00000u) : 0.0f;
  const uint32_t u = reinterpret_cast<const uint16_t*>(v)[at];
  return (u & 0x7F80u) == 0x7F80u ? __uint_as_float(u << 16) : 0.0f;
}

// 16-byte pieces of V that a preparing thread has in flight: as many as its
// registers hold beside the next unit's Q (16 R / 128 pieces).
template <int R>
constexpr int kWidenBatch = R == 16 ? 8 : 4;

// The preparing warps of a CTA: hand out the units (rows[u & 3], q_full[u & 1],
// an empty segment at the end) with their Q, and make V ready tile by tile.
// s_done(g) waits until tile g's scores are done (Q's place is then free),
// o_done(g) until its product is (the widened V's place).
template <int R, int kThreads, bool kFp8, int kLoScale, int kVStages, int kWideRing, class SDone,
          class ODone>
__device__ __forceinline__ void prepare(const TreeArgs& a, const Waits& w, const int* chunk, uint8_t* sq,
                        uint8_t* sv, uint8_t* swide, UnitRows<R>* rows, uint2* row_max,
                        int barrier, uint64_t* q_full, uint64_t* v_full, uint64_t* v_empty,
                        uint64_t* wide_full, int* flagged, int tid, SDone s_done, ODone o_done) {
  const float unit_factor = a.softmax_scale * kLog2e * (kFp8 ? __ldg(a.descale + 1) : 1.0f);
  Walker<R, kThreads> walk;
  walk.init(chunk, gridDim.x);
  Segment seg, next;
  QLoads<R> q;
  bool more = walk.next(a, chunk, next);
  if (more) q.load(a, next, tid, 0);
  int g = 0, tails = 0;
  for (int unit = 0;; ++unit) {
    seg = next;
    if (g > 0) s_done(g - 1);
    // (after an abort somebody may still use the unit that lies there)
    const bool hand_out = !w.any_aborted();
    if (more)
      store_q<R, kFp8, kLoScale>(a, seg, q, sq, rows[unit & 3], row_max, barrier, unit_factor, tid,
                                 hand_out);
    else if (tid == 0 && hand_out)
      rows[unit & 3].seg.t0 = rows[unit & 3].seg.t1 = 0;
    if (hand_out) w.arrive(&q_full[unit & 1]);
    if (!more) return;
    more = walk.next(a, chunk, next);
    if (more) q.load(a, next, tid, 0);
    const int ctx = seg.seq - seg.n;
    for (int t = seg.t0; t < seg.t1; ++t, ++g) {
      const bool tail = t * kTile + kTile > ctx;
      const int vs = g % kVStages;
      bool wild = false;
      w.wait(&v_full[vs], (g / kVStages) & 1);
      if constexpr (kFp8) {
        wild = widen_v<kWidenBatch<R>>(
            sv + vs * 16384, swide + (g % kWideRing) * 32768, tid, tail, t * kTile, ctx, seg.seq,
            [&]() { w.arrive(&v_empty[vs]); },
            [&]() { if (g >= kWideRing) o_done(g - kWideRing); });
      } else if (tail) {
        wild = mend_v(sv + vs * 32768, tid, t * kTile, ctx, seg.seq);
      }
      if (wild) *const_cast<volatile int*>(&flagged[(unit + 1) & 3]) = unit + 1;
      if (kFp8 || tail) {
        const int i = kFp8 ? g : tails++;
        w.arrive(&wide_full[i % kWideRing]);
      }
      if (!kFp8) w.arrive(&v_empty[vs]);   // (the stage's next phase may begin)
    }
  }
}

}  // namespace kv_tree

}  // namespace fp8attn
