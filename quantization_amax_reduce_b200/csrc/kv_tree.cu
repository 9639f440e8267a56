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
//   warp 8      TMA producer: rings of K and V tiles, a box per page (page ids
//               from the block table, one lane per page)
//   warp 9      MMA issuer: S^T(t+1), then O^T += V^T P^T(t)
//   warps 0-3, 4-7: two groups of 128 threads, each with half of the columns:
//               Q into shared memory, V's E4M3 -> f16, softmax, P, epilogue
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
constexpr int kSoftmaxThreads = 256;
constexpr int kThreads = kSoftmaxThreads + 64;
constexpr int kTmaWarp = 8, kMmaWarp = 9;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kPOffset = 8.0f;           // log2 of P at the reference
constexpr float kRefLag = 7.0f;
// A CTA's range is at least this many tiles: below it another CTA and the
// join of its piece cost more than the tiles they save.
constexpr int kMinTiles = 4;

template <int R, bool kFp8>
struct Cfg {
  static constexpr int kHalf = R / 2;                     // columns of a thread
  static constexpr int kN = kFp8 ? 2 * R : R;             // columns of S^T
  static constexpr int kKV = kFp8 ? 16384 : 32768;        // bytes of a K or V tile
  static constexpr int kKStages = kFp8 ? 4 : 3;
  static constexpr int kVStages = kFp8 ? 3 : 2;
  static constexpr int kWide = kFp8 ? 2 * 32768 : 0;      // two f16 V tiles
  static constexpr int kQ = R * 256;                      // hi and lo, or bf16
  static constexpr int kP = kTile * 128;                  // 64 columns of 16 bits
  static constexpr int kSmemData = kKStages * kKV + kVStages * kKV + kWide + kQ + kP;
  static constexpr uint32_t kO = 2 * kN;                  // TMEM column of O^T
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

struct Control {
  uint64_t k_full[4], k_empty[4], v_full[3], v_empty[3];
  uint64_t s_full[2], s_free[2];
  uint64_t q_full, p_full, pv_done, drain;
  uint32_t tmem_base;
  int abort_flag;
  int flagged[2];                        // a node's V of this unit holds Inf or NaN
  int scan[kThreads / 32];
  float factor[2][64];                   // S^T column -> log2 units
  int out_row[2][64];                    // row of `out`, -1 = none
  int node[2][64];
  alignas(16) float red[2][32][4];       // [group][column][warp]
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

// Sums N columns (a power of two up to 32) over the warp's lanes: lane l gets
// the sum of column l % N.
template <int N>
__device__ __forceinline__ float column_sum(float (&v)[N], int lane) {
#pragma unroll
  for (int off = N / 2; off >= 1; off /= 2) {
    const bool up = (lane & off) != 0;
#pragma unroll
    for (int i = 0; i < off; ++i) {
      const float send = up ? v[i] : v[i + off];
      const float mine = up ? v[i + off] : v[i];
      v[i] = mine + __shfl_xor_sync(0xffffffffu, send, off);
    }
  }
#pragma unroll
  for (int off = N; off < 32; off *= 2) v[0] += __shfl_xor_sync(0xffffffffu, v[0], off);
  return v[0];
}

// ---------------------------------------------------------------------------
// Work list: every role walks the same segments (a CTA's tiles of one unit).
// ---------------------------------------------------------------------------

__device__ __forceinline__ int row_tiles(int n, int group, int R) {
  return (n * group + R - 1) / R;
}

// Tiles of the requests before each one into prefix[0..rows]; requests whose
// lengths are inconsistent get none (and set `bad`).  All threads of the CTA.
template <int kCtaThreads>
__device__ void scan_requests(const TreeArgs& a, int R, int32_t* prefix, int* warp_sums,
                              bool* bad) {
  const int per = (a.rows + kCtaThreads - 1) / kCtaThreads;
  const int first = min(a.rows, static_cast<int>(threadIdx.x) * per);
  const int last = min(a.rows, first + per);
  const int64_t held = static_cast<int64_t>(a.width) << a.page_log2;
  auto tiles_of = [&](int b) {
    const int seq = a.seq[b], q0 = a.cu[b], q1 = a.cu[b + 1], n = q1 - q0;
    if (q0 < 0 || q1 < q0 || q1 > a.total_q || n > a.max_q || seq < n || seq > a.max_seqlen ||
        seq > held || (a.mask && n > 64 * a.mask_words)) {
      *bad = true;
      return 0;
    }
    return a.kv_heads * row_tiles(n, a.group, R) * ((seq + kTile - 1) / kTile);
  };
  int sum = 0;
  for (int b = first; b < last; ++b) sum += tiles_of(b);
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
  for (int b = first; b < last; ++b) {
    prefix[b] = at;
    at += tiles_of(b);
  }
  if (threadIdx.x == kCtaThreads - 1) prefix[a.rows] = at;
  __syncthreads();
}

__device__ __forceinline__ int request_of(const int32_t* prefix, int rows, int w) {
  int lo = 0, hi = rows - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (prefix[mid] <= w) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Tiles of a CTA's range.
__device__ __forceinline__ int tiles_per_cta(int total, int ctas) {
  return max(kMinTiles, (total + ctas - 1) / ctas);
}

struct Segment {
  int b, head, rt;       // request, KV head, row tile
  int seq, q0, n;
  int tiles, t0, t1;     // tiles of the unit; this CTA's [t0, t1)
};

struct Walker {
  int w, end, b;
  __device__ __forceinline__ void init(const TreeArgs& a, const int32_t* prefix, int ctas) {
    const int total = prefix[a.rows];
    const int per = tiles_per_cta(total, ctas);
    const int64_t from = static_cast<int64_t>(blockIdx.x) * per;
    w = static_cast<int>(min(from, static_cast<int64_t>(total)));
    end = static_cast<int>(min(from + per, static_cast<int64_t>(total)));
    b = w < end ? request_of(prefix, a.rows, w) : 0;
  }
  __device__ __forceinline__ bool next(const TreeArgs& a, int R, const int32_t* prefix,
                                       Segment& s) {
    if (w >= end) return false;
    while (prefix[b + 1] <= w) ++b;
    s.b = b;
    s.seq = a.seq[b];
    s.q0 = a.cu[b];
    s.n = a.cu[b + 1] - s.q0;
    s.tiles = (s.seq + kTile - 1) / kTile;
    const int rts = row_tiles(s.n, a.group, R);
    const int local = w - prefix[b];
    const int unit = local / s.tiles;
    s.head = unit / rts;
    s.rt = unit - s.head * rts;
    s.t0 = local - unit * s.tiles;
    s.t1 = min(s.tiles, s.t0 + (end - w));
    w += s.t1 - s.t0;
    return true;
  }
};

// ---------------------------------------------------------------------------

template <bool kFp8>
__device__ __forceinline__ float v_value(const uint8_t* p, int64_t i) {
  if (kFp8) return __uint_as_float((p[i] & 0x7Fu) == 0x7Fu ? 0x7FC00000u : 0u);   // NaN or not
  return __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(p)[i]) << 16);
}

template <int R, bool kFp8>
__global__ void __launch_bounds__(kThreads, 1)
kv_tree_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
               const TreeArgs a) {
  using C = Cfg<R, kFp8>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sk = smem;
  uint8_t* sv = sk + C::kKStages * C::kKV;
  uint8_t* swide = sv + C::kVStages * C::kKV;
  uint8_t* sq = swide + C::kWide;
  uint8_t* sp = sq + C::kQ;
  Control& ctl = *reinterpret_cast<Control*>(sp + C::kP);
  int32_t* prefix = reinterpret_cast<int32_t*>(&ctl + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // the join starts as SMs free up; it waits for this grid before it reads
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (threadIdx.x == 0) {
    for (int i = 0; i < 4; ++i) {
      mbar_init(&ctl.k_full[i], 1);
      mbar_init(&ctl.k_empty[i], 1);
    }
    for (int i = 0; i < 3; ++i) {
      mbar_init(&ctl.v_full[i], 1);
      mbar_init(&ctl.v_empty[i], kFp8 ? kSoftmaxThreads / 32 : 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl.s_full[i], 1);
      mbar_init(&ctl.s_free[i], kSoftmaxThreads);
    }
    mbar_init(&ctl.q_full, kSoftmaxThreads);
    mbar_init(&ctl.p_full, kSoftmaxThreads);
    mbar_init(&ctl.pv_done, 1);
    mbar_init(&ctl.drain, 1);
    ctl.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kTmaWarp && lane == 0) {
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&ctl.tmem_base, 512);
    tmem_relinquish();
  }
  bool bad = false;
  scan_requests<kThreads>(a, R, prefix, ctl.scan, &bad);
  if (bad && blockIdx.x == 0) raise_error(a.err, kErrSeqlens);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl.tmem_base;
  const volatile int* abort_flag = &ctl.abort_flag;
  Walker walk;
  walk.init(a, prefix, gridDim.x);
  Segment seg;

  if (warp == kTmaWarp) {
    // ------------------------------------------------------------ producer
    const int page = 1 << a.page_log2;
    const int box = min(page, kTile);
    const int page_rows_log2 = min(a.page_log2, 7);
    int g = 0;
    bool ok = true;
    while (ok && walk.next(a, R, prefix, seg)) {
      const int32_t* table = a.tables + seg.b * a.table_stride;
      // the page of this lane's box of tile t, looked up a tile ahead
      auto look_up = [&](int t) {
        const int key = t * kTile + (lane << page_rows_log2);
        if (lane >= kTile >> page_rows_log2 || key >= seg.seq) return -2;
        return __ldg(table + (key >> a.page_log2));
      };
      int next_id = look_up(seg.t0);
      for (int t = seg.t0; t < seg.t1 && ok; ++t, ++g) {
        const int id = next_id;
        if (t + 1 < seg.t1) next_id = look_up(t + 1);
        const bool load = id != -2;
        if (load && (id < 0 || id >= a.num_pages)) raise_error(a.err, kErrPages);
        const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, load)) * box * (kFp8 ? 128 : 256);
        const int row = a.page_log2 > 7 ? (t * kTile) & (page - 1) : 0;
        const int ks = g % C::kKStages, vs = g % C::kVStages;
        // a page id outside the cache is outside the tensor map: zeros arrive
        if (g >= C::kKStages) ok = mbar_wait(&ctl.k_empty[ks], (g / C::kKStages - 1) & 1, abort_flag);
        if (!ok) break;
        if (lane == 0) mbar_expect_tx(&ctl.k_full[ks], bytes);
        __syncwarp();
        if (load) {
          uint8_t* dst = sk + ks * C::kKV + lane * box * 128;
          tma_load_4d(dst, &tm_k, &ctl.k_full[ks], 0, seg.head, row, id);
          if (!kFp8) tma_load_4d(dst + 16384, &tm_k, &ctl.k_full[ks], 64, seg.head, row, id);
        }
        if (g >= C::kVStages) ok = mbar_wait(&ctl.v_empty[vs], (g / C::kVStages - 1) & 1, abort_flag);
        if (!ok) {
          ++g;   // this tile's K is in flight
          break;
        }
        if (lane == 0) mbar_expect_tx(&ctl.v_full[vs], bytes);
        __syncwarp();
        if (load) {
          uint8_t* dst = sv + vs * C::kKV + lane * box * 128;
          tma_load_4d(dst, &tm_v, &ctl.v_full[vs], 0, seg.head, row, id);
          if (!kFp8) tma_load_4d(dst + 16384, &tm_v, &ctl.v_full[vs], 64, seg.head, row, id);
        }
      }
    }
    if (!ok && lane == 0) {
      ctl.abort_flag = 1;
      raise_error(a.err, kErrTimeout);
    }
    __syncwarp();
    // no copy may still be landing when the CTA leaves (a wait on a V tile
    // that was not issued ends at its limit, after an abort only)
    for (int i = max(0, g - C::kKStages); i < g; ++i)
      mbar_wait(&ctl.k_full[i % C::kKStages], (i / C::kKStages) & 1, nullptr);
    for (int i = max(0, g - C::kVStages); i < g; ++i)
      mbar_wait(&ctl.v_full[i % C::kVStages], (i / C::kVStages) & 1, nullptr);
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA issuer
    const uint32_t id_s = kFp8 ? make_idesc(0, 0, C::kN, 0) : make_idesc(1, 1, C::kN, 0);
    const uint32_t id_pv = make_idesc(kFp8 ? 0 : 1, kFp8 ? 0 : 1, R, 1) | kIdescAMnMajor;
    const uint64_t dk0 = make_sdesc_sw128(smem_u32(sk), 16, 1024);
    const uint64_t dq0 = make_sdesc_sw128(smem_u32(sq), 16, 1024);
    const uint64_t dv0 = make_sdesc_sw128(smem_u32(kFp8 ? swide : sv), 16384, 1024);
    const uint64_t dp0 = make_sdesc_sw128(smem_u32(sp), 16384, 1024);
    auto issue_s = [&](int g) {
      const uint64_t dk = dk0 + static_cast<uint64_t>((g % C::kKStages) * (C::kKV >> 4));
      const uint32_t d = tmem + (g & 1) * C::kN;
      if (elect_one()) {
        if constexpr (kFp8) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) mma_f8_ss(d, dk + 2 * kk, dq0 + 2 * kk, id_s, kk > 0);
        } else {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_bf16_ss(d, dk + (kk >> 2) * 1024 + 2 * (kk & 3),
                        dq0 + (kk >> 2) * (R * 128 >> 4) + 2 * (kk & 3), id_s, kk > 0);
        }
        mma_commit(&ctl.s_full[g & 1]);
        mma_commit(&ctl.k_empty[g % C::kKStages]);
      }
      __syncwarp();
    };
    auto issue_pv = [&](int g, bool first) {
      const uint64_t dv =
          dv0 + static_cast<uint64_t>(kFp8 ? (g & 1) * 2048 : (g % C::kVStages) * 2048);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_bf16_ss(tmem + C::kO, dv + 128 * kk, dp0 + 128 * kk, id_pv, kk > 0 || !first);
        mma_commit(&ctl.pv_done);
        if (!kFp8) mma_commit(&ctl.v_empty[g % C::kVStages]);
      }
      __syncwarp();
    };
    bool ok = true;
    int g = 0, units = 0;      // tiles whose S is issued; segments begun
    bool pending = false, pending_first = false;
    auto finish = [&]() {      // O^T += V^T P^T of tile g - 1
      if (!pending) return;
      const int p = g - 1;
      ok = ok && (kFp8 || mbar_wait(&ctl.v_full[p % C::kVStages], (p / C::kVStages) & 1, abort_flag)) &&
           mbar_wait(&ctl.p_full, p & 1, abort_flag);
      if (ok) {
        tc_fence_after();
        issue_pv(p, pending_first);
      }
      pending = false;
    };
    while (ok && walk.next(a, R, prefix, seg)) {
      // a new unit's Q arrives only after the last unit's epilogue
      finish();
      ok = ok && mbar_wait(&ctl.q_full, units & 1, abort_flag);
      ++units;
      for (int t = seg.t0; t < seg.t1 && ok; ++t) {
        const int ks = g % C::kKStages;
        ok = mbar_wait(&ctl.k_full[ks], (g / C::kKStages) & 1, abort_flag) &&
             (g < 2 || mbar_wait(&ctl.s_free[g & 1], ((g >> 1) - 1) & 1, abort_flag));
        if (!ok) break;
        tc_fence_after();
        issue_s(g);
        finish();
        ++g;
        pending = true;
        pending_first = t == seg.t0;
      }
    }
    finish();
    if (!ok && lane == 0) {
      ctl.abort_flag = 1;
      raise_error(a.err, kErrTimeout);
    }
    __syncwarp();
    // drain: every MMA issued has completed before TMEM is freed
    if (elect_one()) mma_commit(&ctl.drain);
    __syncwarp();
    mbar_wait(&ctl.drain, 0, nullptr);
  } else {
    // ------------------------------------------------------------ softmax
    // After a failed wait (abort) the threads run on without data, so that
    // every named barrier is met, and write nothing.
    const int wg = warp >> 2, wq = warp & 3;
    const int tid = threadIdx.x;
    const int key = 32 * wq + lane;                 // lane of TMEM: key, or channel
    const int bar_wg = 1 + wg;
    const uint32_t lane_off = static_cast<uint32_t>(32 * wq) << 16;
    const uint32_t t_s = tmem + lane_off + wg * C::kHalf;
    const uint32_t t_o = tmem + lane_off + C::kO + wg * C::kHalf;
    const int col0 = wg * C::kHalf;
    uint8_t* prow = sp + (key >> 3) * 1024 + (key & 7) * 128;
    const float unit_factor =
        a.softmax_scale * kLog2e * (kFp8 ? __ldg(a.descale + 1) : 1.0f);
    const float ds_v = kFp8 ? __ldg(a.descale + 2) : 1.0f;
    bool ok = true;
    int g = 0, units = 0;
    while (walk.next(a, R, prefix, seg)) {
      const int par = units & 1;
      const int ctx = seg.seq - seg.n;
      // ---- Q rows of the unit, and what each column stands for
      if (tid == 0) ctl.flagged[par] = 0;
#pragma unroll
      for (int it = 0; it < R * 16 / kSoftmaxThreads; ++it) {
        const int r = it * 16 + (tid >> 4), c = tid & 15;   // row, 8-channel piece
        const int row = seg.rt * R + r;
        const int node = row / a.group, gq = row - node * a.group;
        const bool live = node < seg.n;
        const int head = seg.head * a.group + gq;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (live)
          x = __ldg(reinterpret_cast<const uint4*>(a.q + (seg.q0 + node) * a.q_tok_stride +
                                                   head * a.q_head_stride + c * 8));
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
          auto at = [&](int rr) {
            return sq + (rr >> 3) * 1024 + (rr & 7) * 128 + (((c >> 1) ^ (rr & 7)) << 4) +
                   (c & 1) * 8;
          };
          *reinterpret_cast<uint2*>(at(r)) = make_uint2(hi[0], hi[1]);
          *reinterpret_cast<uint2*>(at(R + r)) = make_uint2(lo[0], lo[1]);
        } else {
          *reinterpret_cast<uint4*>(sq + (c >> 3) * (R * 128) + (r >> 3) * 1024 + (r & 7) * 128 +
                                    (((c & 7) ^ (r & 7)) << 4)) = x;
        }
        if (c == 0) {
          ctl.factor[par][r] = factor;
          ctl.node[par][r] = live ? node : -1;
          ctl.out_row[par][r] = live ? (seg.q0 + node) * (a.kv_heads * a.group) + head : -1;
        }
      }
      fence_proxy_async();
      mbar_arrive(&ctl.q_full);
      group_sync(3, kSoftmaxThreads);
      ++units;

      float off[C::kHalf];      // kPOffset - ref, 0 while unset
      float sum[C::kHalf];
      uint32_t unset = C::kHalf == 32 ? 0xffffffffu : (1u << C::kHalf) - 1;
#pragma unroll
      for (int c = 0; c < C::kHalf; ++c) off[c] = sum[c] = 0.0f;

      auto sees = [&](int c, int j) {   // does column c see node j >= 0?
        const int node = ctl.node[par][col0 + c];
        if (j >= seg.n || node < 0) return false;
        if (!a.mask) return j <= node;
        const unsigned long long word =
            __ldg(a.mask + static_cast<int64_t>(seg.q0 + node) * a.mask_words + (j >> 6));
        return ((word >> (j & 63)) & 1) != 0;
      };

      for (int t = seg.t0; t < seg.t1; ++t, ++g) {
        const int j = t * kTile + key - ctx;            // node of this thread's key, < 0: context
        const bool tail = t * kTile + kTile > ctx;      // the tile holds nodes
        const int vs = g % C::kVStages;
        // ---- V: E4M3 -> f16 (buffer g & 1 is free: its last reader, the
        // product of tile g - 2, was waited for before P of tile g - 1 was
        // written).  In the tail, rows past the sequence become zeros, and so
        // do the non-finite elements of nodes, which a row that does not see
        // the node must not meet as 0 x Inf: the epilogue adds them.
        if constexpr (kFp8) {
          ok = ok && mbar_wait(&ctl.v_full[vs], (g / C::kVStages) & 1, abort_flag);
          const uint8_t* src = sv + vs * C::kKV;
          uint4 x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            x[i] = *reinterpret_cast<const uint4*>(src + (i * 256 + (tid ^ ((tid >> 3) & 7))) * 16);
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl.v_empty[vs]);
          uint8_t* dst = swide + (g & 1) * 32768;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = i * 32 + (tid >> 3), c = tid & 7;   // key, 16-channel piece
            if (tail) {
              const int pos = t * kTile + row;
              if (pos >= seg.seq) {
                x[i] = make_uint4(0, 0, 0, 0);
              } else if (pos >= ctx) {
                uint32_t* w = &x[i].x;
                uint32_t nan = 0;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                  const uint32_t m = __vcmpeq4(w[u] & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
                  w[u] &= ~m;
                  nan |= m;
                }
                if (nan) ctl.flagged[par] = 1;
              }
            }
            uint32_t f[8];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const uint32_t w = (&x[i].x)[u];
              f[2 * u] = cvt_f16x2_from_e4m3x2(w & 0xFFFFu);
              f[2 * u + 1] = cvt_f16x2_from_e4m3x2(w >> 16);
            }
            // channels 16 c .. 16 c + 15: pieces 2 (c & 3), + 1 of half c >> 2;
            // the halves start with different ones (no bank conflicts)
            uint8_t* to = dst + (c >> 2) * 16384 + (row >> 3) * 1024 + (row & 7) * 128;
            const int odd = c >> 2;
            const int p0 = 2 * (c & 3) + odd, p1 = 2 * (c & 3) + (odd ^ 1);
            const uint4 lo = make_uint4(f[0], f[1], f[2], f[3]);
            const uint4 hi = make_uint4(f[4], f[5], f[6], f[7]);
            *reinterpret_cast<uint4*>(to + ((p0 ^ (row & 7)) << 4)) = odd ? hi : lo;
            *reinterpret_cast<uint4*>(to + ((p1 ^ (row & 7)) << 4)) = odd ? lo : hi;
          }
        } else if (tail) {
          ok = ok && mbar_wait(&ctl.v_full[vs], (g / C::kVStages) & 1, abort_flag);
          uint8_t* src = sv + vs * C::kKV;
          for (int i = tid; i < C::kKV / 16; i += kSoftmaxThreads) {
            const int pos = t * kTile + ((i >> 3) & 127);
            if (pos < ctx) continue;
            uint4* p = reinterpret_cast<uint4*>(src + i * 16);
            uint4 x = pos < seg.seq ? *p : make_uint4(0, 0, 0, 0);
            uint32_t* w = &x.x;
            uint32_t wild = pos < seg.seq ? 0u : 1u;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const uint32_t m = __vcmpeq2(w[u] & 0x7F807F80u, 0x7F807F80u);
              w[u] &= ~m;
              wild |= m;
            }
            if (wild) {
              *p = x;
              if (pos < seg.seq) ctl.flagged[par] = 1;
            }
          }
        }

        // ---- scores, in log2 units against the reference
        ok = ok && mbar_wait(&ctl.s_full[g & 1], (g >> 1) & 1, abort_flag);
        tc_fence_after();
        float x[C::kHalf];
        {
          uint32_t u[C::kHalf];
          tmem_ld<C::kHalf>(t_s + (g & 1) * C::kN, u);
          if constexpr (kFp8) {
            uint32_t v[C::kHalf];
            tmem_ld<C::kHalf>(t_s + (g & 1) * C::kN + R, v);
            tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < C::kHalf; ++c)
              x[c] = fmaf(__uint_as_float(v[c]), 0.0625f, __uint_as_float(u[c]));
          } else {
            tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < C::kHalf; ++c) x[c] = __uint_as_float(u[c]);
          }
        }
        tc_fence_before();
        mbar_arrive(&ctl.s_free[g & 1]);
        float top = -INFINITY;
#pragma unroll
        for (int c = 0; c < C::kHalf; ++c) {
          const float f = kFp8 ? ctl.factor[par][col0 + c] : unit_factor;
          x[c] = fmaf(x[c], f, off[c]);
        }
        if (tail) {
#pragma unroll
          for (int c = 0; c < C::kHalf; ++c)
            if (j >= 0 && !sees(c, j)) x[c] = -INFINITY;
        }
#pragma unroll
        for (int c = 0; c < C::kHalf; ++c) top = fmaxf(top, x[c]);

        // ---- does the reference of a column move?
        if (group_any(bar_wg, unset != 0 || top > kPOffset + kRefLag)) {
#pragma unroll
          for (int c = 0; c < C::kHalf; ++c) {
            const float m = warp_max(x[c]);
            if (lane == 0) ctl.red[wg][c][wq] = m;
          }
          group_sync(bar_wg, 128);
          bool rescale = false;
          float scale[C::kHalf];
#pragma unroll
          for (int c = 0; c < C::kHalf; ++c) {
            const float4 m4 = *reinterpret_cast<const float4*>(ctl.red[wg][c]);
            const float m = fmaxf(fmaxf(m4.x, m4.y), fmaxf(m4.z, m4.w));
            const bool fresh = (unset >> c & 1u) != 0;
            scale[c] = 1.0f;
            if (fresh ? m > -INFINITY : m > kPOffset + kRefLag) {
              const float by = kPOffset - m;
              off[c] += by;
              x[c] += by;
              if (!fresh) {
                scale[c] = ex2_approx(by);
                sum[c] *= scale[c];
                rescale = true;
              }
              unset &= ~(1u << c);
            }
          }
          // the same for all 128 threads; an unset column's O^T is zero
          if (rescale) {
            ok = ok && mbar_wait(&ctl.pv_done, (g - 1) & 1, abort_flag);
            tc_fence_after();
            uint32_t o[C::kHalf];
            tmem_ld<C::kHalf>(t_o, o);
            tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < C::kHalf; ++c)
              o[c] = __float_as_uint(__uint_as_float(o[c]) * scale[c]);
            tmem_st<C::kHalf>(t_o, o);
            tmem_st_wait();
          }
          group_sync(bar_wg, 128);   // `red` may be written again
        }

        // ---- P
        uint32_t w[C::kHalf / 2];
#pragma unroll
        for (int c = 0; c < C::kHalf; c += 2) {
          const float p0 = ex2_approx(x[c]), p1 = ex2_approx(x[c + 1]);
          sum[c] += p0;
          sum[c + 1] += p1;
          w[c / 2] = kFp8 ? cvt_f16x2(p0, p1) : cvt_bf16x2(p0, p1);
        }
        if (g > 0) ok = ok && mbar_wait(&ctl.pv_done, (g - 1) & 1, abort_flag);
#pragma unroll
        for (int i = 0; i < C::kHalf / 8; ++i)
          *reinterpret_cast<uint4*>(prow + (((col0 / 8 + i) ^ (key & 7)) << 4)) =
              make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        fence_proxy_async();
        tc_fence_before();
        mbar_arrive(&ctl.p_full);
      }

      // ---- epilogue: lane = channel
      const int n_rows = seg.n * a.group - seg.rt * R;   // live columns of the tile
      const float mine = column_sum<C::kHalf>(sum, lane);
      if (lane < C::kHalf) ctl.red[wg][lane][wq] = mine;
      ok = ok && mbar_wait(&ctl.pv_done, (g - 1) & 1, abort_flag);
      tc_fence_after();
      float o[C::kHalf];
      {
        uint32_t u[C::kHalf];
        tmem_ld<C::kHalf>(t_o, u);
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < C::kHalf; ++c) o[c] = __uint_as_float(u[c]);
      }
      tc_fence_before();
      group_sync(3, kSoftmaxThreads);   // sums and `flagged` are in place
      if (ctl.flagged[par]) {
        const int head = seg.head;
        for (int pos = max(ctx, seg.t0 * kTile); pos < min(seg.seq, seg.t1 * kTile); ++pos) {
          const int id = a.tables[seg.b * a.table_stride + (pos >> a.page_log2)];
          if (id < 0 || id >= a.num_pages) continue;
          const float v = v_value<kFp8>(
              a.v, id * a.page_stride + (pos & ((1 << a.page_log2) - 1)) * a.slot_stride +
                       head * a.head_stride + key);
          if ((__float_as_uint(v) & 0x7F800000u) != 0x7F800000u) continue;
#pragma unroll
          for (int c = 0; c < C::kHalf; ++c)
            if (sees(c, pos - ctx)) o[c] += v;
        }
      }
      const bool live = ok && !*abort_flag;
      if (seg.t0 == 0 && seg.t1 == seg.tiles) {
#pragma unroll
        for (int c = 0; c < C::kHalf; ++c) {
          const float4 s4 = *reinterpret_cast<const float4*>(ctl.red[wg][c]);
          const float l = (s4.x + s4.y) + (s4.z + s4.w);
          const int row = ctl.out_row[par][col0 + c];
          if (live && row >= 0)
            a.out[static_cast<int64_t>(row) * kHeadDim + key] =
                __float2bfloat16(l == 0.0f ? 0.0f : o[c] * (ds_v / l));
        }
      } else {
        const int64_t piece = 2 * static_cast<int64_t>(blockIdx.x) + (seg.t0 == 0);
#pragma unroll
        for (int c = 0; c < C::kHalf; ++c) {
          const float4 s4 = *reinterpret_cast<const float4*>(ctl.red[wg][c]);
          const int64_t at = piece * R + col0 + c;
          if (live && col0 + c < n_rows) {
            a.part_o[at * kHeadDim + key] = o[c];
            if (key == 0)
              a.part_ml[at] = make_float2((unset >> c & 1u) ? -INFINITY : kPOffset - off[c],
                                          (s4.x + s4.y) + (s4.z + s4.w));
          }
        }
      }
    }
    if (!ok) {
      ctl.abort_flag = 1;
      raise_error(a.err, kErrTimeout);
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------------
// Join: block (x, y) takes the unit that crosses from CTA x's range into CTA
// x + 1's, if it starts in CTA x's, and rows 8 y .. 8 y + 7 of it:
// out = sum_i 2^(ref_i - ref) O_i ds_v / sum_i 2^(ref_i - ref) l_i, pieces in
// order.  Bound: launch and latency; the pieces are in L2.
// ---------------------------------------------------------------------------

constexpr int kJoinThreads = 256;
constexpr int kJoinRows = 8;

template <int R, bool kFp8>
__global__ void __launch_bounds__(kJoinThreads) kv_tree_join_kernel(const TreeArgs a, int ctas) {
  extern __shared__ int32_t prefix[];
  __shared__ int warp_sums[kJoinThreads / 32];
  bool bad = false;
  scan_requests<kJoinThreads>(a, R, prefix, warp_sums, &bad);
  const int total = prefix[a.rows];
  const int per = tiles_per_cta(total, ctas);
  const int64_t border = static_cast<int64_t>(blockIdx.x + 1) * per;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (border >= total) return;
  const int w = static_cast<int>(border);
  const int b = request_of(prefix, a.rows, w);
  const int q0 = a.cu[b], n = a.cu[b + 1] - q0, tiles = (a.seq[b] + kTile - 1) / kTile;
  const int rts = row_tiles(n, a.group, R);
  const int unit = (w - prefix[b]) / tiles;
  const int from = prefix[b] + unit * tiles, to = from + tiles;
  const int c0 = from / per, c1 = (to - 1) / per;   // its CTAs
  if (from == w || c0 != static_cast<int>(blockIdx.x)) return;
  const int head = unit / rts, rt = unit - head * rts;
  const float ds_v = kFp8 ? __ldg(a.descale + 2) : 1.0f;
  const int d = threadIdx.x & 127;
  for (int i = threadIdx.x >> 7; i < kJoinRows; i += kJoinThreads / 128) {
    const int r = blockIdx.y * kJoinRows + i;
    const int row = rt * R + r;
    const int node = row / a.group;
    if (node >= n) continue;
    float m = -INFINITY;
    for (int c = c0; c <= c1; ++c)
      m = fmaxf(m, a.part_ml[(2 * static_cast<int64_t>(c) + (c == c0)) * R + r].x);
    float o = 0.0f, l = 0.0f;
    for (int c = c0; c <= c1; ++c) {
      const int64_t at = (2 * static_cast<int64_t>(c) + (c == c0)) * R + r;
      const float2 ml = a.part_ml[at];
      // a piece of no visible key has ref = -inf, O = 0 and l = 0; one whose
      // scores were all NaN has ref = -inf and l = NaN
      const float scale = ml.x == -INFINITY ? 1.0f : exp2f(ml.x - m);
      o = fmaf(scale, a.part_o[at * kHeadDim + d], o);
      l = fmaf(scale, ml.y, l);
    }
    const int64_t out_row = static_cast<int64_t>(q0 + node) * (a.kv_heads * a.group) +
                            head * a.group + (row - node * a.group);
    a.out[out_row * kHeadDim + d] = __float2bfloat16(l == 0.0f ? 0.0f : o * (ds_v / l));
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
  return fn(m, c.fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
            const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kMaxCtas = 148;   // one per SM

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
  const int prefix_bytes = (p.rows + 1) * static_cast<int>(sizeof(int32_t));
  constexpr int kBase = 1024 + C::kSmemData + static_cast<int>(sizeof(Control));
  constexpr int kMost = kBase + (kMaxTreeRows + 1) * static_cast<int>(sizeof(int32_t));
  static_assert(kMost <= 232448, "shared memory of a CTA");
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
                               cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
      if (e != cudaSuccess) return e;
      attr_set |= uint64_t{1} << dev;
    }
  }
  const int ctas = launch_ctas(p.rows, p.max_q, p.max_seqlen, p.heads, p.cache.heads);
  kv_tree_kernel<R, kFp8><<<ctas, kThreads, kBase + prefix_bytes, stream>>>(mk, mv, a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || ctas == 1) return e;
  note_launch();   // the caller counts one launch
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas - 1), R / kJoinRows);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(prefix_bytes);
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
