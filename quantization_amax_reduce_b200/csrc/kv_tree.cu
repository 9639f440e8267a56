// Attention of drafted token trees (or single tokens, or chains) over a paged
// KV cache, on tcgen05 tensor cores.
//
// Request b has n_b new tokens ("nodes"), whose K and V already lie in the
// cache at the last n_b of its seq_b positions.  Node i sees every position of
// the context before them, and node m if bit m of its mask is set (without a
// mask: m <= i).  With G = query heads per KV head, a KV head's query rows are
// r = i G + g.  out = ds_v sum_j p_j v_j / sum_j p_j over the keys a row sees,
// p_j = 2^(s_j c - ref), c = ds_k softmax_scale log2(e); no key: 0.
//
// Keys lie on the lanes.  A work item is a 128-key tile of one (request, KV
// head, tile of R query rows); the products are transposed,
//   S^T [128 keys x rows] = K Q^T          O^T [128 channels x rows] += V^T P^T
// so that the 128 rows of the tensor core's A operand are always full of keys
// (or channels) and only N follows the query rows: a decoding step with 8
// query heads to a KV head pays for 16 columns, not for 128 rows.  A thread
// holds one key and half of the rows: the row sum stays in its registers until
// the unit ends, and the running maximum costs one vote per tile (see below).
//
//   warps 0-3, 4-7: two groups of 128 threads, each with half of the columns:
//               softmax, P, epilogue
//   warps 8, 9  TMA producers of K and of V: rings of tiles, a box per page
//               (page ids from the block table, one lane per page)
//   warp 10     MMA issuer: S^T(t+1), then O^T += V^T P^T(t)
//   warps 11-14 the next unit's Q into shared memory; V: E4M3 -> f16 into the
//               buffer that the product reads, and the rows that must not touch
//               it (past the sequence, non-finite)
// One lane of a warp waits and arrives for it: 256 threads that each try the
// same mbarrier cost some 250 cycles a time.
//
// E4M3 cache: K feeds kind::f8f6f4 as it lies.  A row of Q (bf16), scaled by a
// power of two to [128, 256), is the sum of two E4M3 numbers to 2^-22 of its
// largest element (exactly, for elements above 2^-14 of it): hi, and the
// remainder times 16.  They are two column blocks of the one product
// (N = 2 R), added after it, so nothing of Q is lost.  V is
// widened to f16 (exact) on its way and P is f16, 2^8 at the reference: P in
// E4M3 would cost 2.6 % rms per key, and its 2^-18 range would drop the
// far tail of a long context.  bf16 cache: bf16 products, P bf16.
//
// Reference: ref starts at the first tile's maximum and moves only when a
// score exceeds it by more than 7 (2^15 stays inside f16): then P never
// saturates and O^T is rescaled only on a move.  A tile asks "does any thread
// of the group exceed it?" in one barrier with a vote instead of reducing each
// column over 128 lanes.
//
// Split: the tiles of all units, in order (request, head, row tile, key tile),
// are cut into one equal range per CTA, one CTA per SM, so ragged lengths
// balance without the host knowing them.  A unit that spans CTAs leaves
// (O, ref, sum) of each piece in the workspace, at most two pieces per CTA,
// and a second kernel joins them in order: results do not depend on timing.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "kernels.h"
#include "sm100_ptx.cuh"
#include "state.cuh"

namespace fp8attn {

namespace {

constexpr int kTile = 128;                 // keys of a tile
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kPOffset = 8.0f;           // log2 of P at the reference
constexpr float kRefLag = 7.0f;
// A CTA's range is at least this many tiles: below it another CTA and the
// join of its piece cost more than the tiles they save.
constexpr int kMinTiles = 4;
constexpr int kMaxCtas = 148;              // one per SM

// One CTA per SM, whose stages hold as much in flight as they can: two CTAs of
// half the stages each hid each other's unit switches, but read 3.7 TB/s where
// one with deep rings reads 6.4 (16 columns, E4M3).
template <int R, bool kFp8>
struct Cfg {
  static constexpr int kGroups = 2;
  static constexpr int kCols = R / kGroups;               // columns of a softmax thread
  static constexpr int kSoftmaxWarps = 4 * kGroups, kSoftmaxThreads = 128 * kGroups;
  static constexpr int kTmaWarp = kSoftmaxWarps, kMmaWarp = kTmaWarp + 2;   // K, V; products
  static constexpr int kPrepWarp = kMmaWarp + 1, kPrepWarps = 4;
  static constexpr int kThreads = 32 * (kPrepWarp + kPrepWarps);
  static constexpr int kN = kFp8 ? 2 * R : R;             // columns of S^T
  static constexpr int kKV = kFp8 ? 16384 : 32768;        // bytes of a K or V tile
  static constexpr int kKStages = kFp8 ? (R == 16 ? 5 : 4) : 3;
  static constexpr int kVStages = kFp8 ? (R == 64 ? 3 : 4) : (R == 64 ? 2 : 3);
  static constexpr int kWide = kFp8 ? 2 : 0;              // f16 V tiles of 32 KB
  // Rings of barriers: a waiter tests the parity of the phase it wants, so the
  // phase after it on the same barrier must not end before the waiter passed.
  static constexpr int kSRing = kKStages;
  static constexpr int kPvRing = kFp8 ? kWide : kVStages;
  static constexpr int kWideRing = kFp8 ? kWide : kVStages;
  static constexpr int kQ = R * 256;                      // hi and lo, or bf16
  static constexpr int kPitch = 2 * R;                    // bytes of a key's row of P
  static constexpr int kP = kTile * kPitch;               // = R x 256: O^T is staged there
  static constexpr int kSmemData = (kKStages + kVStages) * kKV + kWide * 32768 + kQ + kP;
  static constexpr uint32_t kO = 2 * kN;                  // TMEM column of O^T
  static constexpr uint32_t kTmem = 512;
};

struct TreeArgs {
  const uint16_t* q;
  int64_t q_tok_stride, q_head_stride;
  const uint8_t* v;                      // V cache, for the non-finite rows
  int64_t page_stride, slot_stride, head_stride;   // elements
  int num_pages, page_log2, kv_heads, group;
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
  int32_t* err;
};

// A CTA's tiles [t0, t1) of one unit.
struct Segment {
  int b, head, rt;       // request, KV head, row tile
  int seq, q0, n;
  int tiles, t0, t1;     // tiles of the unit; this CTA's (none: the end)
};

// What a unit's columns stand for.  Units u and u + 1 may be in use while unit
// u + 2's slot is written.
template <int R>
struct Columns {
  alignas(16) float factor[R];           // S^T -> log2 units
  alignas(16) float off[R];              // kPOffset - ref, 0 while unset
  int out_row[R];                        // row of `out`, -1 = none
  int node[R];                           // -1 = none
  Segment seg;
};

template <int R, bool kFp8>
struct Control {
  using C = Cfg<R, kFp8>;
  // s_full: S^T of a tile is done, for the softmax, and its K stage is free;
  // pv_done: O^T of a tile is done, and P, the widened V and a bf16 V stage
  // are free.  One commit each: a commit costs the issuer as much as a product.
  uint64_t k_full[C::kKStages], s_full[C::kSRing], v_full[C::kVStages], v_empty[C::kVStages];
  uint64_t wide_full[C::kWideRing], pv_done[C::kPvRing];   // wide_full: V is as it is read
  uint64_t q_full[2], p_full, drain;     // q_full: a unit's Q and columns are in place
  uint32_t tmem_base;
  int abort_flag;
  int flagged[4];                        // [u & 3] = u + 1: a node's V of unit u holds Inf or NaN
  int warp_sums[16];
  int chunk[C::kThreads + 1];            // tiles before a thread's requests
  Columns<R> col[4];
  float top[C::kGroups][4][C::kCols];    // [group][warp][column]
  float sum[C::kGroups][4][C::kCols];
  alignas(16) float bc[C::kSoftmaxWarps][2][C::kCols];   // a warp's values, lane -> all lanes
};

__device__ __forceinline__ void raise_error(int32_t* err, uint32_t bits) {
  if (err) atomicOr(reinterpret_cast<unsigned int*>(err), bits);
}

__device__ __forceinline__ void group_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Does any of the group's 128 threads say yes?
__device__ __forceinline__ bool group_any(int id, bool yes) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 q, %1, 0;\n\t"
      "bar.red.or.pred p, %2, 128, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(yes)), "r"(id)
      : "memory");
  return r != 0;
}

template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[N]) {
  if constexpr (N == 8) tmem_ld8(taddr, r);
  else if constexpr (N == 16) tmem_ld16(taddr, r);
  else tmem_ld32(taddr, r);
}

template <int N>
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&r)[N]) {
  if constexpr (N == 8) tmem_st8(taddr, r);
  else if constexpr (N == 16) tmem_st16(taddr, r);
  else tmem_st32(taddr, r);
}

// Reduces N columns (a power of two up to 32) over the warp's lanes: lane l
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
// Work list: every role walks the same segments (a CTA's tiles of one unit).
// ---------------------------------------------------------------------------

struct Request {
  int seq, q0, n, tiles, row_tiles;
  __device__ __forceinline__ int work(int kv_heads) const { return kv_heads * row_tiles * tiles; }
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
  return ok;
}

// chunk[i] = tiles of the requests before thread i's; chunk[kThreads] = all.
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
  for (int w = 0; w < warp; ++w) at += warp_sums[w];
  chunk[threadIdx.x] = at;
  if (threadIdx.x == kThreads - 1) chunk[kThreads] = at + sum;
  return bad;   // (the caller syncs)
}

// The request that a work item belongs to.
template <int R, int kThreads>
struct Finder {
  Request r;
  int b = -1, start = 0, stop = 0;   // request, its first item, end of its chunk
  __device__ __forceinline__ void seek(const TreeArgs& a, const int* chunk, int w) {
    if (b >= 0 && w < start + r.work(a.kv_heads)) return;
    while (b >= 0 && b + 1 < stop) {   // a neighbour of the same chunk
      start += r.work(a.kv_heads);
      read_request<R>(a, ++b, r);
      if (w < start + r.work(a.kv_heads)) return;
    }
    int lo = 0, hi = kThreads - 1;     // the last chunk that starts at or before w
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (chunk[mid] <= w) lo = mid; else hi = mid - 1;
    }
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

// Tiles of a CTA's range.
__device__ __forceinline__ int tiles_per_cta(int total, int ctas) {
  return max(kMinTiles, (total + ctas - 1) / ctas);
}

template <int R, int kThreads>
struct Walker {
  Finder<R, kThreads> find;
  int w, end;
  __device__ __forceinline__ void init(const int* chunk, int ctas) {
    const int total = chunk[kThreads];
    const int per = tiles_per_cta(total, ctas);
    const int64_t from = static_cast<int64_t>(blockIdx.x) * per;
    w = static_cast<int>(min(from, static_cast<int64_t>(total)));
    end = static_cast<int>(min(from + per, static_cast<int64_t>(total)));
  }
  __device__ __forceinline__ bool next(const TreeArgs& a, const int* chunk, Segment& s) {
    if (w >= end) return false;
    find.seek(a, chunk, w);
    const Request& r = find.r;
    s.b = find.b;
    s.seq = r.seq;
    s.q0 = r.q0;
    s.n = r.n;
    s.tiles = r.tiles;
    const int local = w - find.start;
    const int unit = local / r.tiles;
    s.head = unit / r.row_tiles;
    s.rt = unit - s.head * r.row_tiles;
    s.t0 = local - unit * r.tiles;
    s.t1 = min(s.tiles, s.t0 + (end - w));
    w += s.t1 - s.t0;
    return true;
  }
};

// ---------------------------------------------------------------------------

template <int R, bool kFp8>
__global__ void __launch_bounds__(Cfg<R, kFp8>::kThreads, 1)
kv_tree_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
               const TreeArgs a) {
  using C = Cfg<R, kFp8>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sk = smem;
  uint8_t* sv = sk + C::kKStages * C::kKV;
  uint8_t* swide = sv + C::kVStages * C::kKV;
  uint8_t* sq = swide + C::kWide * 32768;
  uint8_t* sp = sq + C::kQ;
  Control<R, kFp8>& ctl = *reinterpret_cast<Control<R, kFp8>*>(sp + C::kP);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // the join starts as SMs free up; it waits for this grid before it reads
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kKStages; ++i) mbar_init(&ctl.k_full[i], 1);
    for (int i = 0; i < C::kSRing; ++i) mbar_init(&ctl.s_full[i], 1);
    for (int i = 0; i < C::kVStages; ++i) {
      mbar_init(&ctl.v_full[i], 1);
      mbar_init(&ctl.v_empty[i], C::kPrepWarps);
    }
    for (int i = 0; i < C::kWideRing; ++i) mbar_init(&ctl.wide_full[i], C::kPrepWarps);
    for (int i = 0; i < C::kPvRing; ++i) mbar_init(&ctl.pv_done[i], 1);
    for (int i = 0; i < 4; ++i) ctl.flagged[i] = 0;
    mbar_init(&ctl.q_full[0], C::kPrepWarps);
    mbar_init(&ctl.q_full[1], C::kPrepWarps);
    mbar_init(&ctl.p_full, C::kSoftmaxWarps);
    mbar_init(&ctl.drain, 1);
    ctl.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == C::kTmaWarp && lane == 0) tma_prefetch_desc(&tm_k);
  if (warp == C::kTmaWarp + 1 && lane == 0) tma_prefetch_desc(&tm_v);
  if (warp == C::kMmaWarp) {
    tmem_alloc(&ctl.tmem_base, C::kTmem);
    tmem_relinquish();
  }
  const bool bad = scan_requests<R, C::kThreads>(a, ctl.chunk, ctl.warp_sums);
  if (bad && blockIdx.x == 0) raise_error(a.err, kErrSeqlens);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl.tmem_base;
  const volatile int* abort_flag = &ctl.abort_flag;
  // A wait that gives up sets the abort flag, which ends all other waits at
  // once; the roles then run on without data (so that every barrier is met)
  // and write no output.  (The whole warp tests: 64 cycles when the phase is
  // over already, against 117 for one lane and a warp sync.)
  auto wait_warp = [&](uint64_t* bar, uint32_t parity) {
    if (!mbar_wait(bar, parity, abort_flag)) {
      if (!*abort_flag) raise_error(a.err, kErrTimeout);
      ctl.abort_flag = 1;
    }
    __syncwarp();
  };
  auto arrive_warp = [&](uint64_t* bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };
  auto wait_pv = [&](int g) { wait_warp(&ctl.pv_done[g % C::kPvRing], (g / C::kPvRing) & 1); };
  // the preparing warps hand out the units, with their Q; a copy ends the loop
  auto unit_at = [&](int unit, Segment& s) {
    wait_warp(&ctl.q_full[unit & 1], (unit >> 1) & 1);
    s = ctl.col[unit & 3].seg;
    return s.t0 < s.t1 && !*abort_flag;
  };

  if (warp < C::kMmaWarp && warp >= C::kTmaWarp) {
    // ------------------------------------------------------------ producers
    // of K (the first warp) and V: neither waits for the other's stages
    const bool is_k = warp == C::kTmaWarp;
    const CUtensorMap* map = is_k ? &tm_k : &tm_v;
    uint8_t* ring = is_k ? sk : sv;
    uint64_t* full = is_k ? ctl.k_full : ctl.v_full;
    const int stages = is_k ? C::kKStages : C::kVStages;
    const int page = 1 << a.page_log2;
    const int box = min(page, kTile);
    const int box_log2 = min(a.page_log2, 7);
    Walker<R, C::kThreads> walk;
    walk.init(ctl.chunk, gridDim.x);
    Segment seg;
    int g = 0, stage = 0, turn = 0;
    while (!*abort_flag && walk.next(a, ctl.chunk, seg)) {
      const int32_t* table = a.tables + seg.b * a.table_stride;
      // the page of this lane's box of tile t, looked up a tile ahead
      auto look_up = [&](int t) {
        const int key = t * kTile + (lane << box_log2);
        if (lane >= kTile >> box_log2 || key >= seg.seq) return -2;
        return __ldg(table + (key >> a.page_log2));
      };
      int next_id = look_up(seg.t0);
      for (int t = seg.t0; t < seg.t1; ++t, ++g) {
        const int id = next_id;
        if (t + 1 < seg.t1) next_id = look_up(t + 1);
        const bool load = id != -2;
        if (is_k && load && (id < 0 || id >= a.num_pages)) raise_error(a.err, kErrPages);
        const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, load)) * box * (kFp8 ? 128 : 256);
        const int row = a.page_log2 > 7 ? (t * kTile) & (page - 1) : 0;
        // a page id outside the cache is outside the tensor map: zeros arrive;
        // after an abort the copies go on, into stages that nobody reads
        if (turn > 0) {
          if (is_k) {        // its S^T frees a K stage
            const int freed = g - C::kKStages;
            wait_warp(&ctl.s_full[freed % C::kSRing], (freed / C::kSRing) & 1);
          } else {           // the preparing warps, and O^T, free a V stage
            wait_warp(&ctl.v_empty[stage], (turn - 1) & 1);
            if (!kFp8) wait_pv(g - C::kVStages);
          }
        }
        if (lane == 0) mbar_expect_tx(&full[stage], bytes);
        __syncwarp();
        if (load) {
          uint8_t* dst = ring + stage * C::kKV + lane * box * 128;
          tma_load_4d(dst, map, &full[stage], 0, seg.head, row, id);
          if (!kFp8) tma_load_4d(dst + 16384, map, &full[stage], 64, seg.head, row, id);
        }
        __syncwarp();
        if (++stage == stages) stage = 0, ++turn;
      }
    }
    // no copy may still be landing when the CTA leaves
    if (lane == 0)
      for (int i = max(0, g - stages); i < g; ++i)
        mbar_wait(&full[i % stages], (i / stages) & 1, nullptr);
    __syncwarp();
  } else if (warp == C::kMmaWarp) {
    // ------------------------------------------------------------ MMA issuer
    // (the whole warp walks, one elected lane issues: descriptors then stay in
    // uniform registers; a lone thread took twice the cycles per product)
    const uint32_t id_s = kFp8 ? make_idesc(0, 0, C::kN, 0) : make_idesc(1, 1, C::kN, 0);
    const uint32_t id_pv = make_idesc(kFp8 ? 0 : 1, kFp8 ? 0 : 1, R, 1) | kIdescAMnMajor;
    const uint64_t dk0 = make_sdesc_sw128(smem_u32(sk), 16, 1024);
    const uint64_t dq0 = make_sdesc_sw128(smem_u32(sq), 16, 1024);
    const uint64_t dv0 = make_sdesc_sw128(smem_u32(kFp8 ? swide : sv), 16384, 1024);
    const uint64_t dp0 = make_sdesc(smem_u32(sp), 16384, 8 * C::kPitch,
                                    R == 16 ? kSwizzle32 : R == 32 ? kSwizzle64 : kSwizzle128);
    Segment seg;
    int g = 0;                 // tiles whose S is issued
    int tails = 0;             // bf16: tiles whose V went through the value warps
    bool pending = false, pending_first = false, pending_tail = false;
    auto finish = [&]() {      // O^T += V^T P^T of tile g - 1
      if (!pending) return;
      const int p = g - 1;
      pending = false;
      if (kFp8 || pending_tail) {
        const int i = kFp8 ? p : tails++;
        wait_warp(&ctl.wide_full[i % C::kWideRing], (i / C::kWideRing) & 1);
      } else {
        wait_warp(&ctl.v_full[p % C::kVStages], (p / C::kVStages) & 1);
      }
      wait_warp(&ctl.p_full, p & 1);
      tc_fence_after();
      const uint64_t dv =
          dv0 + static_cast<uint64_t>((p % (kFp8 ? C::kWide : C::kVStages)) * (32768 >> 4));
      const uint32_t acc0 = pending_first ? 0u : 1u;
      uint64_t ad[8], bd[8];
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        ad[kk] = dv + 128 * kk;          // both MN-major: 16 keys' rows per MMA
        bd[kk] = dp0 + C::kPitch * kk;
      }
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_bf16_ss(tmem + C::kO, ad[kk], bd[kk], id_pv, kk > 0 ? 1u : acc0);
        mma_commit(&ctl.pv_done[p % C::kPvRing]);
      }
      __syncwarp();
    };
    for (int unit = 0;; ++unit) {
      finish();
      if (!unit_at(unit, seg)) break;
      for (int t = seg.t0; t < seg.t1; ++t) {
        const int ks = g % C::kKStages;
        // (the softmax has read S^T of tile g - 2: its P was waited for)
        wait_warp(&ctl.k_full[ks], (g / C::kKStages) & 1);
        tc_fence_after();
        const uint64_t dk = dk0 + static_cast<uint64_t>(ks * (C::kKV >> 4));
        const uint32_t d = tmem + (g & 1) * C::kN;
        constexpr int kSteps = kFp8 ? 4 : 8;
        uint64_t ad[kSteps], bd[kSteps];
#pragma unroll
        for (int kk = 0; kk < kSteps; ++kk) {
          ad[kk] = dk + (kk >> 2) * 1024 + 2 * (kk & 3);
          bd[kk] = dq0 + (kk >> 2) * (R * 128 >> 4) + 2 * (kk & 3);
        }
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < kSteps; ++kk) {
            if (kFp8) mma_f8_ss(d, ad[kk], bd[kk], id_s, kk > 0);
            else mma_bf16_ss(d, ad[kk], bd[kk], id_s, kk > 0);
          }
          mma_commit(&ctl.s_full[g % C::kSRing]);
        }
        __syncwarp();
        finish();
        ++g;
        pending = true;
        pending_first = t == seg.t0;
        pending_tail = t * kTile + kTile > seg.seq - seg.n;
      }
    }
    // drain: every MMA issued has completed before TMEM is freed
    if (elect_one()) mma_commit(&ctl.drain);
    __syncwarp();
    if (lane == 0) mbar_wait(&ctl.drain, 0, nullptr);
    __syncwarp();
  } else if (warp >= C::kPrepWarp) {
    // ------------------------------------------------------------ Q and V
    const int tid = threadIdx.x - C::kPrepWarp * 32;
    const float unit_factor =
        a.softmax_scale * kLog2e * (kFp8 ? __ldg(a.descale + 1) : 1.0f);
    // Q: a half warp per row, 8 channels a lane; loaded a unit ahead
    constexpr int kLoads = R / 8;
    uint4 xq[kLoads];
    auto load_q = [&](const Segment& s) {
#pragma unroll
      for (int it = 0; it < kLoads; ++it) {
        const int row = s.rt * R + it * 8 + (tid >> 4);
        const int node = row / a.group, gq = row - node * a.group;
        xq[it] = make_uint4(0, 0, 0, 0);
        if (node < s.n)
          xq[it] = __ldg(reinterpret_cast<const uint4*>(
              a.q + (s.q0 + node) * a.q_tok_stride +
              (s.head * a.group + gq) * a.q_head_stride + (tid & 15) * 8));
      }
    };
    auto store_q = [&](const Segment& s, Columns<R>& col) {
      const int c = tid & 15;
#pragma unroll
      for (int it = 0; it < kLoads; ++it) {
        const int r = it * 8 + (tid >> 4);
        const uint4 x = xq[it];
        float factor = unit_factor;
        if constexpr (kFp8) {
          const uint32_t w[4] = {x.x, x.y, x.z, x.w};
          uint32_t m = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
          m = max(m & 0xFFFFu, m >> 16);
#pragma unroll
          for (int off = 8; off >= 1; off /= 2) m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
          // 2^e <= amax < 2^(e + 1); 2^(7 - e) and 2^(e - 7) are normal numbers
          const int e = max(static_cast<int>(m >> 7) - 127, -119);
          const float up = __uint_as_float(static_cast<uint32_t>(127 + 7 - e) << 23);
          factor = unit_factor * __uint_as_float(static_cast<uint32_t>(127 + e - 7) << 23);
          const bool whole = m < 0x7F80u;   // a row with Inf or NaN is NaN throughout
          uint32_t hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float x0 = __uint_as_float(w[i] << 16) * up;
            const float x1 = __uint_as_float(w[i] & 0xFFFF0000u) * up;
            const uint32_t h = cvt_e4m3x2(x0, x1);
            const uint32_t hf = cvt_f16x2_from_e4m3x2(h);
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hf));
            const uint32_t l = cvt_e4m3x2((x0 - f.x) * 16.0f, (x1 - f.y) * 16.0f);
            hi[i >> 1] |= (whole ? h : 0x7F7Fu) << (16 * (i & 1));
            lo[i >> 1] |= (whole ? l : 0x7F7Fu) << (16 * (i & 1));
          }
          uint8_t* to = sq + (r >> 3) * 1024 + (r & 7) * 128 + (((c >> 1) ^ (r & 7)) << 4) +
                        (c & 1) * 8;
          *reinterpret_cast<uint2*>(to) = make_uint2(hi[0], hi[1]);
          *reinterpret_cast<uint2*>(to + R * 128) = make_uint2(lo[0], lo[1]);   // row R + r
        } else {
          *reinterpret_cast<uint4*>(sq + (c >> 3) * (R * 128) + (r >> 3) * 1024 + (r & 7) * 128 +
                                    (((c & 7) ^ (r & 7)) << 4)) = x;
        }
        if (c == 0) {
          col.factor[r] = factor;
          col.off[r] = 0.0f;
        }
      }
      if (tid < R) {
        const int row = s.rt * R + tid;
        const int node = row / a.group, gq = row - node * a.group;
        const bool live = node < s.n;
        col.node[tid] = live ? node : -1;
        col.out_row[tid] =
            live ? (s.q0 + node) * (a.kv_heads * a.group) + s.head * a.group + gq : -1;
      }
      if (tid == 0) col.seg = s;
      fence_proxy_async();
    };
    Walker<R, C::kThreads> walk;
    walk.init(ctl.chunk, gridDim.x);
    Segment seg, next;
    bool more = walk.next(a, ctl.chunk, next);
    if (more) load_q(next);
    int g = 0, units = 0, tails = 0;
    for (;;) {
      seg = next;
      // Q's place is free when the last unit's last S^T is done
      if (g > 0) wait_warp(&ctl.s_full[(g - 1) % C::kSRing], ((g - 1) / C::kSRing) & 1);
      if (more) store_q(seg, ctl.col[units & 3]);
      else if (tid == 0) ctl.col[units & 3].seg.t0 = ctl.col[units & 3].seg.t1 = 0;
      arrive_warp(&ctl.q_full[units & 1]);
      if (!more) break;
      more = walk.next(a, ctl.chunk, next);
      if (more) load_q(next);
      // V.  In tiles that hold nodes, rows past the sequence become zeros, and
      // so do the non-finite elements of nodes, which a query that does not
      // see the node must not meet as 0 x Inf: the epilogue adds them.
      const int ctx = seg.seq - seg.n;
      ++units;
      for (int t = seg.t0; t < seg.t1; ++t, ++g) {
        const bool tail = t * kTile + kTile > ctx;
        const int vs = g % C::kVStages;
        uint8_t* src = sv + vs * C::kKV;
        bool wild = false;
        wait_warp(&ctl.v_full[vs], (g / C::kVStages) & 1);
        if (!kFp8 && !tail) {   // nothing to do; the stage's next phase may begin
          arrive_warp(&ctl.v_empty[vs]);
          continue;
        }
        if constexpr (kFp8) {
          constexpr int kRows = C::kPrepWarps * 4;   // rows of one pass of the threads
          uint8_t* wide = swide + (g % C::kWide) * 32768;
          // a thread's pieces of 16 channels: c = tid & 7 of rows kRows i + tid / 8.
          // They become pieces 2 (c & 3) and + 1 of half c >> 2; the halves
          // start with different ones (no bank conflicts).
          const int row = tid >> 3, c = tid & 7, odd = c >> 2;
          uint8_t* to = wide + odd * 16384 + row * 128;
          const int p0 = ((2 * (c & 3) + odd) ^ (row & 7)) << 4;
          const int p1 = ((2 * (c & 3) + (odd ^ 1)) ^ (row & 7)) << 4;
#pragma unroll 1
          for (int i0 = 0; i0 < kTile / kRows; i0 += 8) {
            uint4 x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              x[i] = *reinterpret_cast<const uint4*>(
                  src + ((i0 + i) * kRows * 8 + (tid ^ ((tid >> 3) & 7))) * 16);
            if (i0 + 8 == kTile / kRows) arrive_warp(&ctl.v_empty[vs]);
            if (tail) {
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const int pos = t * kTile + (i0 + i) * kRows + row;
                uint32_t* w = &x[i].x;
                uint32_t nan = 0;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                  const uint32_t m = pos >= seg.seq ? 0xffffffffu
                                     : pos >= ctx   ? __vcmpeq4(w[u] & 0x7F7F7F7Fu, 0x7F7F7F7Fu)
                                                    : 0u;
                  w[u] &= ~m;
                  nan |= m;
                }
                wild |= nan != 0 && pos < seg.seq;
              }
            }
            if (i0 == 0 && g >= C::kWide) wait_pv(g - C::kWide);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              uint32_t f[8];
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                const uint32_t w = (&x[i].x)[u];
                f[2 * u] = cvt_f16x2_from_e4m3x2(w & 0xFFFFu);
                f[2 * u + 1] = cvt_f16x2_from_e4m3x2(w >> 16);
              }
              const uint4 lo = make_uint4(f[0], f[1], f[2], f[3]);
              const uint4 hi = make_uint4(f[4], f[5], f[6], f[7]);
              uint8_t* d = to + (i0 + i) * kRows * 128;
              *reinterpret_cast<uint4*>(d + p0) = odd ? hi : lo;
              *reinterpret_cast<uint4*>(d + p1) = odd ? lo : hi;
            }
          }
        } else {
          for (int i = tid; i < C::kKV / 16; i += 32 * C::kPrepWarps) {
            const int pos = t * kTile + ((i >> 3) & 127);
            if (pos < ctx) continue;
            uint4* p = reinterpret_cast<uint4*>(src + i * 16);
            uint4 x = pos < seg.seq ? *p : make_uint4(0, 0, 0, 0);
            uint32_t* w = &x.x;
            uint32_t m_any = 0;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const uint32_t m = __vcmpeq2(w[u] & 0x7F807F80u, 0x7F807F80u);
              w[u] &= ~m;
              m_any |= m;
            }
            if (m_any || pos >= seg.seq) *p = x;
            wild |= m_any != 0;
          }
        }
        fence_proxy_async();
        if (wild) *const_cast<volatile int*>(&ctl.flagged[units & 3]) = units;
        const int i = kFp8 ? g : tails++;
        arrive_warp(&ctl.wide_full[i % C::kWideRing]);
        if (!kFp8) arrive_warp(&ctl.v_empty[vs]);
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    constexpr int kCols = C::kCols, kPart = kCols < 16 ? kCols : 16;
    const int wg = warp >> 2, wq = warp & 3;
    const int key = 32 * wq + lane;                 // lane of TMEM: key, or channel
    const int bar_wg = 1 + wg;
    const uint32_t lane_off = static_cast<uint32_t>(32 * wq) << 16;
    const uint32_t t_s = tmem + lane_off + wg * kCols;
    const uint32_t t_o = tmem + lane_off + C::kO + wg * kCols;
    const int col0 = wg * kCols;
    const int c_mine = lane & (kCols - 1);          // where a lane stands for a column
    constexpr uint32_t kAll = kCols == 32 ? 0xffffffffu : (1u << kCols) - 1;
    // this key's row of P; 16-byte pieces are swizzled by address bits 7 and up
    uint8_t* prow = sp + key * C::kPitch;
    const int pswz = R == 64 ? key & 7 : R == 32 ? (key >> 1) & 3 : (key >> 2) & 1;
    const float ds_v = kFp8 ? __ldg(a.descale + 2) : 1.0f;
    Segment seg;
    int g = 0;
    for (int unit = 0; unit_at(unit, seg); ++unit) {
      Columns<R>& col = ctl.col[unit & 3];
      const int ctx = seg.seq - seg.n;
      uint64_t sum2[kCols / 2];   // row sums of this thread's keys, columns in pairs
#pragma unroll
      for (int c = 0; c < kCols / 2; ++c) sum2[c] = 0;
      const int my_node = col.node[col0 + c_mine];
      const unsigned long long* my_mask =
          a.mask + static_cast<int64_t>(seg.q0 + max(my_node, 0)) * a.mask_words;
      float my_off = 0.0f;      // kPOffset - ref, 0 while unset
      // live columns that have met no visible key yet
      uint32_t unset = __ballot_sync(0xffffffffu, my_node >= 0) & kAll;

      for (int t = seg.t0; t < seg.t1; ++t, ++g) {
        // ---- which columns see this thread's key: lane c collects column c's
        // bits for the warp's 32 keys, then the warp transposes
        const bool tail = t * kTile + kTile > ctx;      // the tile holds nodes
        uint32_t sees = kAll;
        if (tail) {
          const int j0 = t * kTile + 32 * wq - ctx;     // node of the warp's first key
          uint32_t bits = j0 < 0 ? low_bits(-j0) : 0;
          if (my_node >= 0 && j0 > -32 && j0 < seg.n) {
            uint32_t m;
            if (a.mask)
              m = mask_bits(my_mask, a.mask_words, j0) & low_bits(seg.n - j0);
            else
              m = my_node < j0 ? 0u : low_bits(my_node - j0 + 1);
            bits |= m;
          }
          sees = transpose_bits(bits, lane);
        }

        // ---- scores, in log2 units against the reference
        wait_warp(&ctl.s_full[g % C::kSRing], (g / C::kSRing) & 1);
        tc_fence_after();
        // columns in pairs: x2[c / 2] = columns c, c + 1
        uint64_t x2[kCols / 2];
        {
          const uint64_t sixteenth = f2_pack(0.0625f, 0.0625f);
#pragma unroll
          for (int h = 0; h < kCols; h += kPart) {
            uint32_t u[kPart], v[kPart];
            tmem_ld<kPart>(t_s + (g & 1) * C::kN + h, u);
            if (kFp8) tmem_ld<kPart>(t_s + (g & 1) * C::kN + R + h, v);
            tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < kPart; c += 4) {
              const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(&col.factor[col0 + h + c]);
              const ulonglong2 o = *reinterpret_cast<const ulonglong2*>(&col.off[col0 + h + c]);
              uint64_t lo = f2_bits(u[c], u[c + 1]), hi = f2_bits(u[c + 2], u[c + 3]);
              if (kFp8) {
                lo = f2_fma(f2_bits(v[c], v[c + 1]), sixteenth, lo);
                hi = f2_fma(f2_bits(v[c + 2], v[c + 3]), sixteenth, hi);
              }
              x2[(h + c) / 2] = f2_fma(lo, f.x, o.x);
              x2[(h + c) / 2 + 1] = f2_fma(hi, f.y, o.y);
            }
          }
        }
        float x[kCols];
#pragma unroll
        for (int c = 0; c < kCols; c += 2) f2_unpack(x2[c / 2], x[c], x[c + 1]);
        if (tail) {
#pragma unroll
          for (int c = 0; c < kCols; ++c)
            if (!(sees >> c & 1u)) x[c] = -INFINITY;
        }
        float top = -INFINITY;
        {
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int c = 0; c < kCols; c += 2) m4[(c / 2) & 3] = fmax3(m4[(c / 2) & 3], x[c], x[c + 1]);
          top = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        }

        // ---- does the reference of a column move?
        if (group_any(bar_wg, unset != 0 || top > kPOffset + kRefLag)) {
          float v[kCols];
#pragma unroll
          for (int c = 0; c < kCols; ++c) v[c] = x[c];
          const float mine = reduce_columns<kCols, true>(v, lane);
          if (lane < kCols) ctl.top[wg][wq][lane] = mine;
          group_sync(bar_wg, 128);
          // lane c decides for column c; all four warps come to the same
          const float m = fmaxf(fmaxf(ctl.top[wg][0][c_mine], ctl.top[wg][1][c_mine]),
                                fmaxf(ctl.top[wg][2][c_mine], ctl.top[wg][3][c_mine]));
          const bool fresh = (unset >> c_mine & 1u) != 0;
          const bool moves = fresh ? m > -INFINITY : m > kPOffset + kRefLag;
          const float by = moves ? kPOffset - m : 0.0f;
          const uint32_t moved = __ballot_sync(0xffffffffu, moves) & kAll;
          my_off += by;
          if (lane < kCols) {
            col.off[col0 + lane] = my_off;
            ctl.bc[warp][0][lane] = by;
            ctl.bc[warp][1][lane] = fresh ? 1.0f : ex2_approx(by);
          }
          __syncwarp();
          const bool rescale = (moved & ~unset) != 0;   // an unset column's O^T is zero
          unset &= ~moved;
#pragma unroll
          for (int c = 0; c < kCols; c += 4) {
            const float4 b4 = *reinterpret_cast<const float4*>(&ctl.bc[warp][0][c]);
            const float4 s4 = *reinterpret_cast<const float4*>(&ctl.bc[warp][1][c]);
            x[c] += b4.x, x[c + 1] += b4.y, x[c + 2] += b4.z, x[c + 3] += b4.w;
            sum2[c / 2] = f2_mul(sum2[c / 2], f2_pack(s4.x, s4.y));
            sum2[c / 2 + 1] = f2_mul(sum2[c / 2 + 1], f2_pack(s4.z, s4.w));
          }
          if (rescale) {
            wait_pv(g - 1);
            tc_fence_after();
            uint32_t o[kCols];
            tmem_ld<kCols>(t_o, o);
            tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < kCols; ++c)
              o[c] = __float_as_uint(__uint_as_float(o[c]) * ctl.bc[warp][1][c]);
            tmem_st<kCols>(t_o, o);
            tmem_st_wait();
          }
          __syncwarp();   // `bc` may be written again
        }

        // ---- P
        uint32_t w[kCols / 2];
#pragma unroll
        for (int c = 0; c < kCols; c += 2) {
          const float p0 = ex2_approx(x[c]), p1 = ex2_approx(x[c + 1]);
          sum2[c / 2] = f2_add(sum2[c / 2], f2_pack(p0, p1));
          w[c / 2] = kFp8 ? cvt_f16x2(p0, p1) : cvt_bf16x2(p0, p1);
        }
        if (g > 0) wait_pv(g - 1);
#pragma unroll
        for (int i = 0; i < kCols / 8; ++i)
          *reinterpret_cast<uint4*>(prow + (((col0 / 8 + i) ^ pswz) << 4)) =
              make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        fence_proxy_async();
        tc_fence_before();
        arrive_warp(&ctl.p_full);
      }

      // ---- epilogue: lane = channel
      float sum[kCols];
#pragma unroll
      for (int c = 0; c < kCols; c += 2) f2_unpack(sum2[c / 2], sum[c], sum[c + 1]);
      const float mine = reduce_columns<kCols, false>(sum, lane);
      if (lane < kCols) ctl.sum[wg][wq][lane] = mine;
      wait_pv(g - 1);
      tc_fence_after();
      float o[kCols];
      {
        uint32_t u[kCols];
        tmem_ld<kCols>(t_o, u);
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < kCols; ++c) o[c] = __uint_as_float(u[c]);
      }
      tc_fence_before();
      group_sync(bar_wg, 128);   // the sums are in place
      if (*const_cast<volatile int*>(&ctl.flagged[(unit + 1) & 3]) == unit + 1) {
        for (int pos = max(ctx, seg.t0 * kTile); pos < min(seg.seq, seg.t1 * kTile); ++pos) {
          const int id = a.tables[seg.b * a.table_stride + (pos >> a.page_log2)];
          if (id < 0 || id >= a.num_pages) continue;
          const int64_t at = id * a.page_stride +
                             (pos & ((1 << a.page_log2) - 1)) * a.slot_stride +
                             seg.head * a.head_stride + key;
          const int j = pos - ctx;
          const bool mine_sees =
              my_node >= 0 &&
              (a.mask ? (__ldg(my_mask + (j >> 6)) >> (j & 63) & 1) != 0 : j <= my_node);
          const uint32_t who = __ballot_sync(0xffffffffu, mine_sees);
          float v = 0.0f;
          if (kFp8) {
            if ((a.v[at] & 0x7Fu) == 0x7Fu) v = __uint_as_float(0x7FC00000u);
          } else {
            const uint32_t u = reinterpret_cast<const uint16_t*>(a.v)[at];
            if ((u & 0x7F80u) == 0x7F80u) v = __uint_as_float(u << 16);
          }
#pragma unroll
          for (int c = 0; c < kCols; ++c)
            if (who >> c & 1u) o[c] += v;
        }
      }
      const float l = (ctl.sum[wg][0][c_mine] + ctl.sum[wg][1][c_mine]) +
                      (ctl.sum[wg][2][c_mine] + ctl.sum[wg][3][c_mine]);
      if (seg.t0 == 0 && seg.t1 == seg.tiles) {
        // through shared memory (P's place): rows of 256 bytes, 16 bytes a thread
        if (lane < kCols) ctl.bc[warp][0][lane] = l == 0.0f ? 0.0f : ds_v / l;
        __syncwarp();
        uint8_t* stage = sp + col0 * 256;
#pragma unroll
        for (int c = 0; c < kCols; c += 4) {
          const float4 s4 = *reinterpret_cast<const float4*>(&ctl.bc[warp][0][c]);
          const float sc[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
          for (int u = 0; u < 4; ++u)
            reinterpret_cast<__nv_bfloat16*>(stage + (c + u) * 256)[key] =
                __float2bfloat16(sc[u] == 0.0f ? 0.0f : o[c + u] * sc[u]);
        }
        // (the whole group: its threads are 32 wq + lane = key)
        group_sync(bar_wg, 128);
        if (!*abort_flag) {
#pragma unroll
          for (int it = 0; it < kCols / 8; ++it) {
            const int r = it * 8 + (key >> 4), c = key & 15;
            const int row = col.out_row[col0 + r];
            if (row >= 0)
              reinterpret_cast<uint4*>(a.out + static_cast<int64_t>(row) * kHeadDim)[c] =
                  *reinterpret_cast<const uint4*>(stage + r * 256 + c * 16);
          }
        }
        group_sync(3, C::kSoftmaxThreads);   // P may be written again
      } else if (!*abort_flag) {
        const int64_t piece = (2 * static_cast<int64_t>(blockIdx.x) + (seg.t0 == 0)) * R + col0;
        const int live = seg.n * a.group - seg.rt * R - col0;   // live columns of this group
        float* to = a.part_o + piece * kHeadDim + key;
#pragma unroll
        for (int c = 0; c < kCols; ++c)
          if (c < live) to[c * kHeadDim] = o[c];
        if (wq == 0 && lane < kCols && lane < live)
          a.part_ml[piece + lane] =
              make_float2((unset >> lane & 1u) ? -INFINITY : kPOffset - my_off, l);
      }
      __syncwarp();   // `bc` may be written again
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == C::kMmaWarp) tmem_dealloc(tmem, C::kTmem);
}

// ---------------------------------------------------------------------------
// Join: block (x, y) takes the unit that crosses from CTA x's range into CTA
// x + 1's, if it starts in CTA x's, and rows 8 y .. 8 y + 7 of it:
// out = sum_i 2^(ref_i - ref) O_i ds_v / sum_i 2^(ref_i - ref) l_i, pieces in
// order.  Bound: launch and latency; the pieces are in L2.
// ---------------------------------------------------------------------------

constexpr int kJoinThreads = 256;
constexpr int kJoinRows = kJoinThreads / 32;

template <int R, bool kFp8>
__global__ void __launch_bounds__(kJoinThreads) kv_tree_join_kernel(const TreeArgs a, int ctas) {
  __shared__ int chunk[kJoinThreads + 1];
  __shared__ int warp_sums[kJoinThreads / 32];
  __shared__ float s_scale[kJoinRows][kMaxCtas];
  __shared__ float s_inv[kJoinRows];
  // everything up to the wait needs the lengths alone
  scan_requests<R, kJoinThreads>(a, chunk, warp_sums);
  __syncthreads();
  const int total = chunk[kJoinThreads];
  const int per = tiles_per_cta(total, ctas);
  const int64_t border = static_cast<int64_t>(blockIdx.x + 1) * per;
  Finder<R, kJoinThreads> find;
  const Request& q = find.r;
  const int w = static_cast<int>(min(border, static_cast<int64_t>(total)));
  int unit = 0, c0 = -1, c1 = -1;     // the unit at the border, and its CTAs
  if (w < total) {
    find.seek(a, chunk, w);
    unit = (w - find.start) / q.tiles;
    const int from = find.start + unit * q.tiles;
    if (from < w) {
      c0 = from / per;
      c1 = (from + q.tiles - 1) / per;
    }
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (c0 != static_cast<int>(blockIdx.x)) return;   // none, or an earlier border's
  const int head = unit / q.row_tiles, rt = unit - head * q.row_tiles;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pieces = c1 - c0 + 1;
  // piece i of row r; the first CTA's piece is its last one, the others' their first
  auto at = [&](int i, int r) {
    return (2 * static_cast<int64_t>(c0 + i) + (i == 0)) * R + blockIdx.y * kJoinRows + r;
  };
  // a warp per row: the pieces' weights
  {
    float m = -INFINITY;
    for (int i = lane; i < pieces; i += 32) m = fmaxf(m, a.part_ml[at(i, warp)].x);
#pragma unroll
    for (int off = 16; off >= 1; off /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    float l = 0.0f;
    for (int i = lane; i < pieces; i += 32) {
      const float2 ml = a.part_ml[at(i, warp)];
      // a piece of no visible key has ref = -inf, O = 0 and l = 0; one whose
      // scores were all NaN has ref = -inf and l = NaN
      const float scale = ml.x == -INFINITY ? 1.0f : exp2f(ml.x - m);
      s_scale[warp][i] = scale;
      l = fmaf(scale, ml.y, l);
    }
#pragma unroll
    for (int off = 16; off >= 1; off /= 2) l += __shfl_xor_sync(0xffffffffu, l, off);
    if (lane == 0) s_inv[warp] = l == 0.0f ? 0.0f : (kFp8 ? __ldg(a.descale + 2) : 1.0f) / l;
  }
  __syncthreads();
  const int d = threadIdx.x & 127;
  for (int r = threadIdx.x >> 7; r < kJoinRows; r += kJoinThreads / 128) {
    const int row = rt * R + blockIdx.y * kJoinRows + r;
    const int node = row / a.group;
    if (node >= q.n) continue;
    float o = 0.0f;
#pragma unroll 8
    for (int i = 0; i < pieces; ++i)
      o = fmaf(s_scale[r][i], a.part_o[at(i, r) * kHeadDim + d], o);
    const int64_t out_row = static_cast<int64_t>(q.q0 + node) * (a.kv_heads * a.group) +
                            head * a.group + (row - node * a.group);
    const float inv = s_inv[r];
    a.out[out_row * kHeadDim + d] = __float2bfloat16(inv == 0.0f ? 0.0f : o * inv);
  }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static const EncodeTiledFn fn = []() -> EncodeTiledFn {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<EncodeTiledFn>(f);
    return nullptr;
  }();
  return fn;
}

// (channel, head, row of a page, page); a box is one head's rows of a page (at
// most a tile's 128), 128 bytes of channels, 128-byte swizzle.
bool make_cache_map(CUtensorMap* m, const void* base, const PagedCache& c) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t esz = c.fp8 ? 1 : 2;
  const cuuint64_t page = cuuint64_t{1} << c.page_log2;
  cuuint64_t dims[4] = {128, static_cast<cuuint64_t>(c.heads), page,
                        static_cast<cuuint64_t>(c.num_pages)};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(c.head_stride) * esz,
                           static_cast<cuuint64_t>(c.slot_stride) * esz,
                           static_cast<cuuint64_t>(c.page_stride) * esz};
  cuuint32_t box[4] = {static_cast<cuuint32_t>(c.fp8 ? 128 : 64), 1,
                       static_cast<cuuint32_t>(page < kTile ? page : kTile), 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  // a 128-byte row of a token-major E4M3 page has another head's beside it,
  // which this CTA does not read: no promotion past it
  const bool beside = c.fp8 && c.slot_stride != kHeadDim;
  return fn(m, c.fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
            const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B,
            beside ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}


// Query rows of a tile: the fewest columns that hold a request's rows of a KV
// head (16 is the smallest N; above 64 a request takes several row tiles).
int tile_rows(int max_q, int heads, int kv_heads) {
  const int64_t rows = static_cast<int64_t>(max_q) * (heads / kv_heads);
  return rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
}

int launch_ctas(int rows, int max_q, int max_seqlen, int heads, int kv_heads) {
  const int64_t tiles = kv_tree_max_tiles(rows, max_q, max_seqlen, heads, kv_heads);
  const int64_t ctas = (tiles + kMinTiles - 1) / kMinTiles;
  return static_cast<int>(ctas < 1 ? 1 : ctas < kMaxCtas ? ctas : kMaxCtas);
}

template <int R, bool kFp8>
cudaError_t launch_t(const KvTreeLaunch& p, const TreeArgs& a, cudaStream_t stream) {
  using C = Cfg<R, kFp8>;
  CUtensorMap mk, mv;
  if (!make_cache_map(&mk, p.cache.k, p.cache) || !make_cache_map(&mv, p.cache.v, p.cache))
    return cudaErrorInvalidValue;
  constexpr int kSmem = 1024 + C::kSmemData + static_cast<int>(sizeof(Control<R, kFp8>));
  static_assert(kSmem <= 232448, "shared memory of a CTA");
  static std::mutex mu;
  static uint64_t attr_set = 0;   // bit d: done on device d (one per instantiation)
  {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (!(attr_set >> dev & 1u)) {
      e = cudaFuncSetAttribute(kv_tree_kernel<R, kFp8>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
      if (e != cudaSuccess) return e;
      attr_set |= uint64_t{1} << dev;
    }
  }
  const int ctas = launch_ctas(p.rows, p.max_q, p.max_seqlen, p.heads, p.cache.heads);
  kv_tree_kernel<R, kFp8><<<ctas, C::kThreads, kSmem, stream>>>(mk, mv, a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || ctas == 1) return e;
  note_launch();   // the caller counts one launch
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas - 1), R / kJoinRows);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv_tree_join_kernel<R, kFp8>, a, ctas);
}

}  // namespace

int64_t kv_tree_max_tiles(int rows, int max_q, int max_seqlen, int heads, int kv_heads) {
  const int R = tile_rows(max_q, heads, kv_heads);
  const int64_t row_tiles = (static_cast<int64_t>(max_q) * (heads / kv_heads) + R - 1) / R;
  return row_tiles * kv_heads * rows * ((static_cast<int64_t>(max_seqlen) + kTile - 1) / kTile);
}

size_t kv_tree_workspace_bytes(int rows, int max_q, int max_seqlen, int heads, int kv_heads) {
  const int ctas = launch_ctas(rows, max_q, max_seqlen, heads, kv_heads);
  if (ctas <= 1) return 0;
  return static_cast<size_t>(2 * ctas) * tile_rows(max_q, heads, kv_heads) *
         (kHeadDim * sizeof(float) + sizeof(float2));
}

cudaError_t launch_kv_tree(const KvTreeLaunch& p, cudaStream_t stream) {
  TreeArgs a;
  a.q = static_cast<const uint16_t*>(p.q);
  a.q_tok_stride = p.q_tok_stride;
  a.q_head_stride = p.q_head_stride;
  a.v = static_cast<const uint8_t*>(p.cache.v);
  a.page_stride = p.cache.page_stride;
  a.slot_stride = p.cache.slot_stride;
  a.head_stride = p.cache.head_stride;
  a.num_pages = p.cache.num_pages;
  a.page_log2 = p.cache.page_log2;
  a.kv_heads = p.cache.heads;
  a.group = p.heads / p.cache.heads;
  a.tables = p.tables;
  a.table_stride = p.table_stride;
  a.width = p.width;
  a.seq = p.seq;
  a.cu = p.cu;
  a.rows = p.rows;
  a.max_q = p.max_q;
  a.max_seqlen = p.max_seqlen;
  a.total_q = static_cast<int>(p.total_q);
  a.descale = p.descale;
  a.mask = reinterpret_cast<const unsigned long long*>(p.mask);
  a.mask_words = p.mask_words;
  a.softmax_scale = p.softmax_scale;
  a.out = static_cast<__nv_bfloat16*>(p.out);
  a.err = p.err;
  const int R = tile_rows(p.max_q, p.heads, p.cache.heads);
  const int ctas = launch_ctas(p.rows, p.max_q, p.max_seqlen, p.heads, p.cache.heads);
  a.part_o = static_cast<float*>(p.workspace);
  a.part_ml = reinterpret_cast<float2*>(a.part_o + static_cast<size_t>(2 * ctas) * R * kHeadDim);
  if (p.cache.fp8)
    return R == 16   ? launch_t<16, true>(p, a, stream)
           : R == 32 ? launch_t<32, true>(p, a, stream)
                     : launch_t<64, true>(p, a, stream);
  return R == 16   ? launch_t<16, false>(p, a, stream)
         : R == 32 ? launch_t<32, false>(p, a, stream)
                   : launch_t<64, false>(p, a, stream);
}

}  // namespace fp8attn
