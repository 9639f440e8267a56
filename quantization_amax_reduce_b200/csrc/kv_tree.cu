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
// Up to 32 query rows of a KV head (decoding, small trees), keys lie on the
// lanes.  A work item is a 128-key tile of one (request, KV head, tile of R
// query rows); the products are transposed,
//   S^T [128 keys x rows] = K Q^T          O^T [128 channels x rows] += V^T P^T
// so that the 128 rows of the tensor core's A operand are always full of keys
// (or channels) and only N follows the query rows: a decoding step with 8
// query heads to a KV head pays for 16 columns, not for 128 rows.  With more
// rows the second kernel below lays rows on the lanes.  A thread
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
// A warp waits on a barrier as a whole, and one lane arrives for it: 256
// threads that each arrive cost some 250 cycles a time.
//
// E4M3 cache: K feeds kind::f8f6f4 as it lies.  A row of Q (bf16), scaled by a
// power of two (its tile's, where the rows are within 2^4 of each other) to
// [8, 256), is the sum of two E4M3 numbers to 2^-17 of its largest element
// (exactly, for elements above 2^-9 of it): hi, and the remainder times 16.
// They are two column blocks of the one product (N = 2 R), added after it, so
// nothing of Q is lost.  V is
// widened to f16 (exact) on its way and P is f16, 2^8 at the reference: P in
// E4M3 would cost 2.6 % rms per key, and its 2^-18 range would drop the
// far tail of a long context.  A P below 2^-25, 2^-33 of the reference, becomes
// 0.  Error against 64 bits 1.7e-3 of the result, which is what rounding the
// output to bf16 costs by itself.  bf16 cache: bf16 products, and P in bf16,
// since a product's two operands have one type and bf16 V does not fit f16's
// range: 2.2e-3.  Row sums are fp32 sums of P before its rounding: a key's
// weight is off by that rounding, 2^-11 of it (f16) or 2^-8 (bf16) at most.
//
// Reference: ref starts at the first tile's maximum and moves only when a
// score exceeds it by more than 7 (2^15 stays inside f16): then P never
// saturates and O^T is rescaled only on a move.  A tile asks "does any thread
// of the group exceed it?" in one barrier with a vote instead of reducing each
// column over 128 lanes.
//
// Split: the tiles of all units, in order (request, head, row tile, key tile),
// and a few more a unit for what it costs by itself, are cut into one equal
// range per CTA, one CTA per SM, so ragged lengths balance without the host
// knowing them.  A unit that spans CTAs leaves
// (O, ref, sum) of each piece in the workspace, at most two pieces per CTA,
// and a second kernel joins them in order: results do not depend on timing.
//
// Bound: HBM for long contexts.  8 requests x 32768 tokens, 8 KV heads: E4M3
// with 8 query rows a head 91 us (5.9 TB/s, 0.90 of a copy's rate), with 32 112
// us; bf16 with 8 rows 169 us (6.4 TB/s, 0.97).  For short contexts the latency
// of a unit's stages, some 6000 cycles: 128 chains of 4 over 5 to 300 tokens, 16
// heads, 60 us where the bytes take 25.  A call starts and joins in about 10 us.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>
#include <type_traits>

#include "kernels.h"
#include "kv_tree.cuh"

namespace fp8attn {

namespace {

using namespace kv_tree;

// ---------------------------------------------------------------------------
// Keys on the lanes
// ---------------------------------------------------------------------------

// One CTA per SM, whose stages hold as much in flight as they can: two CTAs of
// half the stages each hid each other's unit switches, but read 3.7 TB/s where
// one with deep rings reads 6.4 (16 columns, E4M3).
template <int R, bool kFp8>
struct KeysCfg {
  static_assert(R == 16 || R == 32, "columns of a tile");
  static constexpr int kGroups = 2;
  static constexpr int kCols = R / kGroups;               // columns of a softmax thread
  static constexpr int kSoftmaxWarps = 4 * kGroups, kSoftmaxThreads = 128 * kGroups;
  static constexpr int kTmaWarp = kSoftmaxWarps, kMmaWarp = kTmaWarp + 2;   // K, V; products
  static constexpr int kPrepWarp = kMmaWarp + 1;
  static constexpr int kThreads = 32 * (kPrepWarp + kPrepWarps);
  static constexpr int kN = kFp8 ? 2 * R : R;             // columns of S^T
  static constexpr int kKV = kFp8 ? 16384 : 32768;        // bytes of a K or V tile
  static constexpr int kKStages = kFp8 ? (R == 16 ? 5 : 4) : 3;
  static constexpr int kVStages = kFp8 ? 4 : 3;
  static constexpr int kWide = kFp8 ? 2 : 0;              // f16 V tiles of 32 KB
  static constexpr int kLoScale = 16;                     // of Q's remainders
  // The stage that a product reads V from, its barrier, and the one that says
  // that V is ready.  A waiter tests the parity of the phase it wants, so the
  // phase after it on the same barrier must not end before the waiter passed.
  static constexpr int kPvRing = kFp8 ? kWide : kVStages;
  static constexpr int kQ = R * 256;                      // hi and lo, or bf16
  static constexpr int kPitch = 2 * R;                    // bytes of a key's row of P
  static constexpr int kP = kTile * kPitch;               // = R x 256: O^T is staged there
  static constexpr int kSmemData = (kKStages + kVStages) * kKV + kWide * 32768 + kQ + kP;
  static constexpr uint32_t kO = 2 * kN;                  // TMEM column of O^T
};

template <int R, bool kFp8>
struct KeysControl {
  using C = KeysCfg<R, kFp8>;
  // s_full: S^T of a tile is done, for the softmax, and its K stage is free;
  // pv_done: O^T of a tile is done, and P, the widened V and a bf16 V stage
  // are free.  One commit each: a commit costs the issuer as much as a product.
  uint64_t k_full[C::kKStages], s_full[C::kKStages], v_full[C::kVStages], v_empty[C::kVStages];
  uint64_t wide_full[C::kPvRing], pv_done[C::kPvRing];   // wide_full: V is as it is read
  uint64_t q_full[2], p_full, drain;     // q_full: a unit's Q and rows are in place
  uint32_t tmem_base;
  int abort_flag;
  int flagged[4];                        // [u & 3] = u + 1: a node's V of unit u holds Inf or NaN
  int warp_sums[32];
  uint2 row_max[kPrepWarps];
  int chunk[C::kThreads + 1];            // tiles before a thread's requests
  UnitRows<R> rows[4];
  float top[C::kGroups][4][C::kCols];    // [group][warp][column]
  float sum[C::kGroups][4][C::kCols];
  alignas(16) float bc[C::kSoftmaxWarps][2][C::kCols];   // a warp's values, lane -> all lanes
};

template <int R, bool kFp8>
__global__ void __launch_bounds__(KeysCfg<R, kFp8>::kThreads, 1)
kv_tree_keys_kernel(const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const TreeArgs a) {
  using C = KeysCfg<R, kFp8>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sk = smem;
  uint8_t* sv = sk + C::kKStages * C::kKV;
  uint8_t* swide = sv + C::kVStages * C::kKV;
  uint8_t* sq = swide + C::kWide * 32768;
  uint8_t* sp = sq + C::kQ;
  KeysControl<R, kFp8>& ctl = *reinterpret_cast<KeysControl<R, kFp8>*>(sp + C::kP);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // the join starts as SMs free up; it waits for this grid before it reads
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kKStages; ++i) {
      mbar_init(&ctl.k_full[i], 1);
      mbar_init(&ctl.s_full[i], 1);
    }
    for (int i = 0; i < C::kVStages; ++i) {
      mbar_init(&ctl.v_full[i], 1);
      mbar_init(&ctl.v_empty[i], kPrepWarps);
    }
    for (int i = 0; i < C::kPvRing; ++i) {
      mbar_init(&ctl.wide_full[i], kPrepWarps);
      mbar_init(&ctl.pv_done[i], 1);
    }
    for (int i = 0; i < 4; ++i) ctl.flagged[i] = 0;
    mbar_init(&ctl.q_full[0], kPrepWarps);
    mbar_init(&ctl.q_full[1], kPrepWarps);
    mbar_init(&ctl.p_full, C::kSoftmaxWarps);
    mbar_init(&ctl.drain, 1);
    ctl.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == C::kTmaWarp && lane == 0) tma_prefetch_desc(&tm_k);
  if (warp == C::kTmaWarp + 1 && lane == 0) tma_prefetch_desc(&tm_v);
  if (warp == C::kMmaWarp) {
    tmem_alloc(&ctl.tmem_base, 512);
    tmem_relinquish();
  }
  const bool bad = scan_requests<R, C::kThreads>(a, ctl.chunk, ctl.warp_sums);
  if (bad && blockIdx.x == 0) raise_error(a.err, kErrSeqlens);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl.tmem_base;
  const Waits w{&ctl.abort_flag, a.err, lane};
  auto wait_pv = [&](int g) { w.wait(&ctl.pv_done[g % C::kPvRing], (g / C::kPvRing) & 1); };
  // whether there is such a unit; the preparing warps have handed it out then
  auto unit_at = [&](int unit) {
    w.wait(&ctl.q_full[unit & 1], (unit >> 1) & 1);
    const Segment& s = ctl.rows[unit & 3].seg;
    return s.t0 < s.t1 && !w.aborted();
  };

  if (warp == C::kTmaWarp) {
    produce<R, C::kThreads, kFp8>(a, w, ctl.chunk, &tm_k, true, sk, C::kKStages, ctl.k_full,
                                  ctl.s_full, nullptr);
  } else if (warp == C::kTmaWarp + 1) {
    produce<R, C::kThreads, kFp8>(a, w, ctl.chunk, &tm_v, false, sv, C::kVStages, ctl.v_full,
                                  ctl.v_empty, kFp8 ? nullptr : ctl.pv_done);
  } else if (warp == C::kMmaWarp) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp walks, one elected lane issues; what comes from shared
    // memory goes through a shuffle, which tells the compiler that it is the
    // same in all lanes, so that descriptors are made in uniform registers.
    const uint32_t id_s = kFp8 ? make_idesc(0, 0, C::kN, 0) : make_idesc(1, 1, C::kN, 0);
    const uint32_t id_pv = make_idesc(kFp8 ? 0 : 1, kFp8 ? 0 : 1, R, 1) | kIdescAMnMajor;
    const uint64_t dk0 = make_sdesc_sw128(smem_u32(sk), 16, 1024);
    const uint64_t dq0 = make_sdesc_sw128(smem_u32(sq), 16, 1024);
    const uint64_t dv0 = make_sdesc_sw128(smem_u32(kFp8 ? swide : sv), 16384, 1024);
    const uint64_t dp0 =
        make_sdesc(smem_u32(sp), 16384, 8 * C::kPitch, R == 16 ? kSwizzle32 : kSwizzle64);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    int ks = 0, k_turn = 0;    // K stage of the next S^T, and its phase
    int s_buf = 0;             // its half of TMEM
    int vs = 0, v_turn = 0;    // V stage of the next product, and its phase
    int p_turn = 0;            // phase of P
    int tails = 0;             // bf16: tiles whose V went through the preparing warps
    auto issue_s = [&]() {
      w.wait(&ctl.k_full[ks], k_turn);
      tc_fence_after();
      const uint64_t dk = dk0 + static_cast<uint64_t>(ks * (C::kKV >> 4));
      const uint32_t d = tm + s_buf * C::kN;
      constexpr int kSteps = kFp8 ? 4 : 8;
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < kSteps; ++kk) {
          const uint64_t ad = dk + (kk >> 2) * 1024 + 2 * (kk & 3);
          const uint64_t bd = dq0 + (kk >> 2) * (R * 128 >> 4) + 2 * (kk & 3);
          if (kFp8) mma_f8_ss(d, ad, bd, id_s, kk > 0);
          else mma_bf16_ss(d, ad, bd, id_s, kk > 0);
        }
        mma_commit(&ctl.s_full[ks]);
      }
      __syncwarp();
      s_buf ^= 1;
      if (++ks == C::kKStages) ks = 0, k_turn ^= 1;
    };
    auto issue_pv = [&](bool first, bool tail, int steps) {
      if (kFp8) {
        w.wait(&ctl.wide_full[vs], v_turn);
      } else if (tail) {
        w.wait(&ctl.wide_full[tails % C::kPvRing], (tails / C::kPvRing) & 1);
        ++tails;
      } else {
        w.wait(&ctl.v_full[vs], v_turn);
      }
      w.wait(&ctl.p_full, p_turn);
      tc_fence_after();
      const uint64_t dv = dv0 + static_cast<uint64_t>(vs * (32768 >> 4));
      const uint32_t acc0 = first ? 0u : 1u;
      if (elect_one()) {
        auto step = [&](int kk) {        // both MN-major: 16 keys' rows per MMA
          mma_bf16_ss(tm + C::kO, dv + 128 * kk, dp0 + C::kPitch * kk, id_pv, kk > 0 ? 1u : acc0);
        };
        if (steps >= 8) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) step(kk);
        } else {
#pragma unroll 1
          for (int kk = 0; kk < steps; ++kk) step(kk);
        }
        mma_commit(&ctl.pv_done[vs]);
      }
      __syncwarp();
      p_turn ^= 1;
      if (++vs == C::kPvRing) vs = 0, v_turn ^= 1;
    };
    for (int unit = 0;; ++unit) {
      const bool go = unit_at(unit);
      const Segment& seg = ctl.rows[unit & 3].seg;
      if (!__shfl_sync(0xffffffffu, static_cast<int>(go), 0)) break;
      const int n = __shfl_sync(0xffffffffu, seg.t1 - seg.t0, 0);
      // tiles from this one on hold nodes
      const int tail0 = __shfl_sync(0xffffffffu, (seg.seq - seg.n) / kTile - seg.t0, 0);
      // groups of 16 keys from this tile on, so that the last stops at the sequence's end
      const int groups = __shfl_sync(0xffffffffu, (seg.seq - seg.t0 * kTile + 15) / 16, 0);
      // S^T runs a tile ahead; the softmax has read the S^T two tiles back
      // when its P is waited for
      issue_s();
      for (int t = 0; t < n; ++t) {
        if (t + 1 < n) issue_s();
        issue_pv(t == 0, t >= tail0, groups - 8 * t);
      }
    }
    // drain: every MMA issued has completed before TMEM is freed
    if (elect_one()) mma_commit(&ctl.drain);
    __syncwarp();
    if (lane == 0) mbar_wait(&ctl.drain, 0, nullptr);
    __syncwarp();
  } else if (warp >= C::kPrepWarp) {
    prepare<R, C::kThreads, kFp8, C::kLoScale, C::kVStages, C::kPvRing>(
        a, w, ctl.chunk, sq, sv, swide, ctl.rows, ctl.row_max, 2 + C::kGroups, ctl.q_full,
        ctl.v_full, ctl.v_empty, ctl.wide_full, ctl.flagged, threadIdx.x - 32 * C::kPrepWarp,
        [&](int g) { w.wait(&ctl.s_full[g % C::kKStages], (g / C::kKStages) & 1); }, wait_pv);
  } else {
    // ------------------------------------------------------------ softmax
    constexpr int kCols = C::kCols;
    const int wg = warp >> 2, wq = warp & 3;
    const int key = 32 * wq + lane;                 // lane of TMEM: key, or channel
    const int bar_wg = 1 + wg;
    const uint32_t lane_off = static_cast<uint32_t>(32 * wq) << 16;
    const uint32_t t_s = tmem + lane_off + wg * kCols;
    const uint32_t t_o = tmem + lane_off + C::kO + wg * kCols;
    const int col0 = wg * kCols;
    const int c_mine = lane & (kCols - 1);          // where a lane stands for a column
    constexpr uint32_t kAll = (1u << kCols) - 1;
    // this key's row of P; 16-byte pieces are swizzled by address bits 7 and up
    uint8_t* prow = sp + key * C::kPitch;
    const int pswz = R == 32 ? (key >> 1) & 3 : (key >> 2) & 1;
    const float ds_v = kFp8 ? __ldg(a.descale + 2) : 1.0f;
    if (threadIdx.x == 0 && a.join) a.join[blockIdx.x] = {0, 0, 0, 0, 0};
    int g = 0;
    // (all softmax warps share barriers in a unit: they agree to begin it)
    for (int unit = 0; !group_any(1 + C::kGroups, C::kSoftmaxThreads, !unit_at(unit)); ++unit) {
      const UnitRows<R>& col = ctl.rows[unit & 3];
      const Segment& seg = col.seg;   // (in shared memory: registers are short)
      if (threadIdx.x == 0 && seg.t0 == 0 && seg.t1 < seg.tiles)
        a.join[blockIdx.x] = join_info(seg, tree_items_per_cta(ctl.chunk[C::kThreads], gridDim.x));
      const int ctx = seg.seq - seg.n;
      // columns in pairs: row sums of this thread's keys; kPOffset - ref, 0 while unset
      uint64_t sum2[kCols / 2], off2[kCols / 2];
#pragma unroll
      for (int c = 0; c < kCols / 2; ++c) sum2[c] = off2[c] = 0;
      const float factor = col.factor[0];
      const bool one_factor = col.one_factor != 0;
      const int my_node = col.node[col0 + c_mine];
      const unsigned long long* my_mask =
          a.mask + static_cast<int64_t>(seg.q0 + max(my_node, 0)) * a.mask_words;
      float my_off = 0.0f;      // kPOffset - ref, 0 while unset
      // live columns that have met no visible key yet
      const uint32_t live = __ballot_sync(0xffffffffu, my_node >= 0) & kAll;
      uint32_t unset = live;
      const int row0 = seg.rt * R + col0;

      for (int t = seg.t0; t < seg.t1; ++t, ++g) {
        // ---- which columns see this thread's key.  A chain: column c is row
        // row0 + c, of node (row0 + c) / group, so columns from j group - row0
        // on.  A tree: lane c collects column c's bits for the warp's 32 keys,
        // then the warp transposes.
        const bool tail = t * kTile + kTile > ctx;      // the tile holds nodes
        uint32_t sees = kAll;
        if (tail && !a.mask) {
          const int j = t * kTile + key - ctx;
          if (j >= 0)
            sees = j < seg.n ? live & ~low_bits(max(0, min(32, j * a.group - row0))) : 0u;
        } else if (tail) {
          const int j0 = t * kTile + 32 * wq - ctx;     // node of the warp's first key
          uint32_t bits = j0 < 0 ? low_bits(-j0) : 0;
          if (my_node >= 0 && j0 > -32 && j0 < seg.n)
            bits |= mask_bits(my_mask, a.mask_words, j0) & low_bits(seg.n - j0);
          sees = transpose_bits(bits, lane);
        }

        // ---- scores, in log2 units against the reference
        w.wait(&ctl.s_full[g % C::kKStages], (g / C::kKStages) & 1);
        tc_fence_after();
        // columns in pairs: x2[c / 2] = columns c, c + 1
        uint64_t x2[kCols / 2];
        {
          const uint64_t sixteenth = f2_pack(0.0625f, 0.0625f);
          uint32_t u[kCols], v[kCols];
          tmem_ld<kCols>(t_s + (g & 1) * C::kN, u);
          if (kFp8) tmem_ld<kCols>(t_s + (g & 1) * C::kN + R, v);
          tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < kCols; c += 2) {
            x2[c / 2] = f2_bits(u[c], u[c + 1]);
            if (kFp8) x2[c / 2] = f2_fma(f2_bits(v[c], v[c + 1]), sixteenth, x2[c / 2]);
          }
          if (!kFp8 || one_factor) {
            const uint64_t f2 = f2_pack(factor, factor);
#pragma unroll
            for (int c = 0; c < kCols / 2; ++c) x2[c] = f2_fma(x2[c], f2, off2[c]);
          } else {
#pragma unroll
            for (int c = 0; c < kCols / 2; ++c)
              x2[c] = f2_fma(x2[c], *reinterpret_cast<const uint64_t*>(&col.factor[col0 + 2 * c]),
                             off2[c]);
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
        if (group_any(bar_wg, 128, unset != 0 || top > kPOffset + kRefLag)) {
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
            off2[c / 2] = f2_add(off2[c / 2], f2_pack(b4.x, b4.y));
            off2[c / 2 + 1] = f2_add(off2[c / 2 + 1], f2_pack(b4.z, b4.w));
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
        uint32_t pw[kCols / 2];
#pragma unroll
        for (int c = 0; c < kCols; c += 2) {
          const float p0 = ex2_approx(x[c]), p1 = ex2_approx(x[c + 1]);
          sum2[c / 2] = f2_add(sum2[c / 2], f2_pack(p0, p1));
          pw[c / 2] = kFp8 ? cvt_f16x2(p0, p1) : cvt_bf16x2(p0, p1);
        }
        if (g > 0) wait_pv(g - 1);
#pragma unroll
        for (int i = 0; i < kCols / 8; ++i)
          *reinterpret_cast<uint4*>(prow + (((col0 / 8 + i) ^ pswz) << 4)) =
              make_uint4(pw[4 * i], pw[4 * i + 1], pw[4 * i + 2], pw[4 * i + 3]);
        fence_proxy_async();
        tc_fence_before();
        w.arrive(&ctl.p_full);
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
          const float v = wild_value<kFp8>(a.v, at);
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
        if (!w.aborted()) {
#pragma unroll
          for (int it = 0; it < kCols / 8; ++it) {
            const int r = it * 8 + (key >> 4), c = key & 15;
            const int row = col.out_row[col0 + r];
            if (row >= 0)
              reinterpret_cast<uint4*>(a.out + static_cast<int64_t>(row) * kHeadDim)[c] =
                  *reinterpret_cast<const uint4*>(stage + r * 256 + c * 16);
          }
        }
        group_sync(1 + C::kGroups, C::kSoftmaxThreads);   // P may be written again
      } else if (!w.aborted()) {
        const int64_t piece = (2 * static_cast<int64_t>(blockIdx.x) + (seg.t0 == 0)) * R + col0;
        float* to = a.part_o + piece * kHeadDim + key;
#pragma unroll
        for (int c = 0; c < kCols; ++c)
          if (live >> c & 1u) to[c * kHeadDim] = o[c];
        if (wq == 0 && lane < kCols && (live >> lane & 1u))
          a.part_ml[piece + lane] =
              make_float2((unset >> lane & 1u) ? -INFINITY : kPOffset - my_off, l);
      }
      __syncwarp();   // `bc` may be written again
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == C::kMmaWarp) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------------
// Rows on the lanes: more than 32 query rows of a KV head
//
// S [128 rows x 128 keys] = Q K^T, O [128 rows x 128 channels] += P V: a thread
// holds a query row, so its maximum, sum, mask and rescaling are its own.  The
// two softmax groups take alternate tiles of a unit, each with its own scores,
// O, reference and sum, so that one's exponentials run beside the other's
// products; they are joined like two pieces when the unit ends.  Up to 64 rows
// lie on the lanes twice, and the second copies take the second half of each
// tile's keys (their P is zero in the other half): half the exponentials a
// thread, at the same products.  P lies in
// TMEM over the first half of its scores, and feeds the product from there.
// (The loops over 32 columns stay rolled: a CTA runs a unit's code once or
// twice, and unrolled it waits for its instructions.)
// A tile's scores are read once: its maximum, in a pass of its own, only for a
// row's first reference (before: 8 requests of 4100 and 64 nodes 63.4 us, now
// 60.8).
// Bound: the chain product, softmax, product of a group (about 4300 cycles a tile
// and group, of which the tensor pipe works 2 x 1024 for both groups and the
// exponentials, 16384 a tile at 16 a cycle, as long): 8 requests x 32768 tokens,
// 8 KV heads, E4M3: 64 rows 132 us, 128 rows 158 us (870 TFLOP/s); bf16 178 us
// (HBM, 6.0 TB/s) and 188 us.
// ---------------------------------------------------------------------------

template <bool kFp8>
struct RowsCfg {
  static constexpr int kSoftmaxWarps = 8, kSoftmaxThreads = 256;
  static constexpr int kTmaWarp = kSoftmaxWarps, kMmaWarp = kTmaWarp + 2;   // K, V; products
  static constexpr int kPrepWarp = kMmaWarp + 1;
  static constexpr int kThreads = 32 * (kPrepWarp + kPrepWarps);
  static constexpr int kKV = kFp8 ? 16384 : 32768;
  static constexpr int kKStages = 3;
  static constexpr int kVStages = kFp8 ? 3 : 2;
  static constexpr int kWide = kFp8 ? 2 : 0;
  // Q's remainders go into the same accumulator, unscaled, and each row has its
  // own scale: hi + lo is exact for elements above 2^-9 of the row's largest,
  // and off by 2^-17 of that at most.
  static constexpr int kLoScale = 1;
  static constexpr int kQ = 32768;
  static constexpr int kSmemData = (kKStages + kVStages) * kKV + kWide * 32768 + kQ;
  // TMEM: scores of group i at 128 i, O at 256 + 128 i
  static constexpr uint32_t kO = 256;
};

template <bool kFp8>
struct RowsControl {
  using C = RowsCfg<kFp8>;
  uint64_t k_full[C::kKStages], k_empty[C::kKStages], v_full[C::kVStages], v_empty[C::kVStages];
  // per group (tile parity); pv_done also frees the widened V and a bf16 V stage
  uint64_t s_full[2], p_full[2], pv_done[2], wide_full[2];
  uint64_t q_full[2], drain;
  uint32_t tmem_base;
  int abort_flag;
  int flagged[4];
  int warp_sums[32];
  uint2 row_max[kPrepWarps];
  int chunk[C::kThreads + 1];
  UnitRows<128> rows[4];
  float2 ml[2][128];                     // {ref, sum} of each group's part of a row
  float half[2][64][33];                 // 32 channels of the second copies' parts
};

template <bool kFp8>
__global__ void __launch_bounds__(RowsCfg<kFp8>::kThreads, 1)
kv_tree_rows_kernel(const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const TreeArgs a) {
  using C = RowsCfg<kFp8>;
  constexpr int R = 128;
  static_assert(kFp8 ? C::kWide == 2 : C::kVStages == 2, "pv_done frees by tile parity");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sk = smem;
  uint8_t* sv = sk + C::kKStages * C::kKV;
  uint8_t* swide = sv + C::kVStages * C::kKV;
  uint8_t* sq = swide + C::kWide * 32768;
  RowsControl<kFp8>& ctl = *reinterpret_cast<RowsControl<kFp8>*>(sq + C::kQ);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kKStages; ++i) {
      mbar_init(&ctl.k_full[i], 1);
      mbar_init(&ctl.k_empty[i], 1);
    }
    for (int i = 0; i < C::kVStages; ++i) {
      mbar_init(&ctl.v_full[i], 1);
      mbar_init(&ctl.v_empty[i], kPrepWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl.s_full[i], 1);
      mbar_init(&ctl.p_full[i], 4);
      mbar_init(&ctl.pv_done[i], 1);
      mbar_init(&ctl.wide_full[i], kPrepWarps);
      mbar_init(&ctl.q_full[i], kPrepWarps);
    }
    for (int i = 0; i < 4; ++i) ctl.flagged[i] = 0;
    mbar_init(&ctl.drain, 1);
    ctl.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == C::kTmaWarp && lane == 0) tma_prefetch_desc(&tm_k);
  if (warp == C::kTmaWarp + 1 && lane == 0) tma_prefetch_desc(&tm_v);
  if (warp == C::kMmaWarp) {
    tmem_alloc(&ctl.tmem_base, 512);
    tmem_relinquish();
  }
  const bool bad = scan_requests<R, C::kThreads>(a, ctl.chunk, ctl.warp_sums);
  if (bad && blockIdx.x == 0) raise_error(a.err, kErrSeqlens);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl.tmem_base;
  const Waits w{&ctl.abort_flag, a.err, lane};
  auto wait_pv = [&](int g) { w.wait(&ctl.pv_done[g & 1], (g >> 1) & 1); };
  // whether there is such a unit; the preparing warps have handed it out then
  auto unit_at = [&](int unit) {
    w.wait(&ctl.q_full[unit & 1], (unit >> 1) & 1);
    const Segment& s = ctl.rows[unit & 3].seg;
    return s.t0 < s.t1 && !w.aborted();
  };

  if (warp == C::kTmaWarp) {
    produce<R, C::kThreads, kFp8>(a, w, ctl.chunk, &tm_k, true, sk, C::kKStages, ctl.k_full,
                                  ctl.k_empty, nullptr);
  } else if (warp == C::kTmaWarp + 1) {
    produce<R, C::kThreads, kFp8>(a, w, ctl.chunk, &tm_v, false, sv, C::kVStages, ctl.v_full,
                                  ctl.v_empty, kFp8 ? nullptr : ctl.pv_done);
  } else if (warp == C::kMmaWarp) {
    // ------------------------------------------------------------ MMA issuer
    const uint32_t id_s = kFp8 ? make_idesc(0, 0, 128, 0) : make_idesc(1, 1, 128, 0);
    const uint32_t id_pv = make_idesc(kFp8 ? 0 : 1, kFp8 ? 0 : 1, 128, 1);
    const uint64_t dq0 = make_sdesc_sw128(smem_u32(sq), 16, 1024);
    const uint64_t dk0 = make_sdesc_sw128(smem_u32(sk), 16, 1024);
    const uint64_t dv0 = make_sdesc_sw128(smem_u32(kFp8 ? swide : sv), 16384, 1024);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    int ks = 0, k_turn = 0;    // K stage of the next scores, and its phase
    int s_side = 0;            // their group
    int side = 0, turn = 0;    // group of the next product, and its phase
    int tails = 0;             // bf16: tiles whose V went through the preparing warps
    auto issue_s = [&]() {
      w.wait(&ctl.k_full[ks], k_turn);
      tc_fence_after();
      const uint64_t dk = dk0 + static_cast<uint64_t>(ks * (C::kKV >> 4));
      const uint32_t d = tm + 128 * s_side;
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          // E4M3: Q's hi tile, then its remainders, against the same K
          const uint64_t ad = dq0 + (kk >> 2) * 1024 + 2 * (kk & 3);
          const uint64_t bd = dk + (kFp8 ? 0 : (kk >> 2) * 1024) + 2 * (kk & 3);
          if (kFp8) mma_f8_ss(d, ad, bd, id_s, kk > 0);
          else mma_bf16_ss(d, ad, bd, id_s, kk > 0);
        }
        mma_commit(&ctl.s_full[s_side]);
        mma_commit(&ctl.k_empty[ks]);
      }
      __syncwarp();
      s_side ^= 1;
      if (++ks == C::kKStages) ks = 0, k_turn ^= 1;
    };
    auto issue_pv = [&](bool first, bool tail, int steps) {
      if (kFp8) {
        w.wait(&ctl.wide_full[side], turn);
      } else if (tail) {
        w.wait(&ctl.wide_full[tails & 1], (tails >> 1) & 1);
        ++tails;
      } else {
        w.wait(&ctl.v_full[side], turn);
      }
      w.wait(&ctl.p_full[side], turn);
      tc_fence_after();
      const uint64_t dv = dv0 + static_cast<uint64_t>(side * (32768 >> 4));
      const uint32_t p = tm + 128 * side, o = tm + C::kO + 128 * side;
      const uint32_t acc0 = first ? 0u : 1u;
      if (elect_one()) {
        auto step = [&](int kk) {        // 16 keys: 8 columns of P, 16 rows of V
          mma_bf16_ts(o, p + 8 * kk, dv + 128 * kk, id_pv, kk > 0 ? 1u : acc0);
        };
        if (steps >= 8) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) step(kk);
        } else {
#pragma unroll 1
          for (int kk = 0; kk < steps; ++kk) step(kk);
        }
        mma_commit(&ctl.pv_done[side]);
      }
      __syncwarp();
      side ^= 1;
      if (side == 0) turn ^= 1;
    };
    for (int unit = 0;; ++unit) {
      const bool go = unit_at(unit);
      const Segment& seg = ctl.rows[unit & 3].seg;
      if (!__shfl_sync(0xffffffffu, static_cast<int>(go), 0)) break;
      const int n = __shfl_sync(0xffffffffu, seg.t1 - seg.t0, 0);
      const int tail0 = __shfl_sync(0xffffffffu, (seg.seq - seg.n) / kTile - seg.t0, 0);
      // groups of 16 keys from this tile on, so that the last stops at the sequence's end
      const int groups = __shfl_sync(0xffffffffu, (seg.seq - seg.t0 * kTile + 15) / 16, 0);
      // a group's next scores overwrite its P: they follow its product
      issue_s();
      if (n > 1) issue_s();
      for (int t = 0; t < n; ++t) {
        issue_pv(t < 2, t >= tail0, groups - 8 * t);
        if (t + 2 < n) issue_s();
      }
    }
    if (elect_one()) mma_commit(&ctl.drain);
    __syncwarp();
    if (lane == 0) mbar_wait(&ctl.drain, 0, nullptr);
    __syncwarp();
  } else if (warp >= C::kPrepWarp) {
    prepare<R, C::kThreads, kFp8, C::kLoScale, C::kVStages, 2>(
        a, w, ctl.chunk, sq, sv, swide, ctl.rows, ctl.row_max, 4, ctl.q_full, ctl.v_full,
        ctl.v_empty, ctl.wide_full, ctl.flagged, threadIdx.x - 32 * C::kPrepWarp,
        [&](int g) { w.wait(&ctl.k_empty[g % C::kKStages], (g / C::kKStages) & 1); }, wait_pv);
  } else {
    // ------------------------------------------------------------ softmax
    const int wg = warp >> 2, wq = warp & 3;
    const int row = 32 * wq + lane;
    const uint32_t lane_off = static_cast<uint32_t>(32 * wq) << 16;
    const uint32_t t_s = tmem + lane_off + 128 * wg;
    const uint32_t t_o = tmem + lane_off + C::kO + 128 * wg;
    const float ds_v = kFp8 ? __ldg(a.descale + 2) : 1.0f;
    if (threadIdx.x == 0 && a.join) a.join[blockIdx.x] = {0, 0, 0, 0, 0};
    int g = 0;
    for (int unit = 0; !group_any(1, C::kSoftmaxThreads, !unit_at(unit)); ++unit) {
      const UnitRows<R>& rows = ctl.rows[unit & 3];
      const Segment& seg = rows.seg;   // (in shared memory: registers are short)
      if (threadIdx.x == 0 && seg.t0 == 0 && seg.t1 < seg.tiles)
        a.join[blockIdx.x] = join_info(seg, tree_items_per_cta(ctl.chunk[C::kThreads], gridDim.x));
      const int ctx = seg.seq - seg.n;
      // (not zero: a hidden score is -inf before it is multiplied)
      const float factor = rows.factor[row] == 0.0f ? 1.17549435e-38f : rows.factor[row];
      const int node = rows.node[row];
      const unsigned long long* mask =
          a.mask + static_cast<int64_t>(seg.q0 + max(node, 0)) * a.mask_words;
      // node's view of 32 keys from position pos on
      auto sees = [&](int pos) {
        const int j0 = pos - ctx;
        uint32_t bits = j0 < 0 ? low_bits(-j0) : 0;
        if (node >= 0 && j0 > -32 && j0 < seg.n)
          bits |= a.mask ? mask_bits(mask, a.mask_words, j0) & low_bits(seg.n - j0)
                         : node < j0 ? 0u : low_bits(node - j0 + 1);
        return bits;
      };
      float off = 0.0f;         // kPOffset - ref
      bool set = false;         // whether the row has met a visible key
      uint64_t sum2[2] = {0, 0};
      const int g0 = g;
      // the 32-key columns of a tile that this row takes
      const bool doubled = is_doubled<R>(a, seg);
      const int h0 = doubled ? wq & 2 : 0, h1 = doubled ? h0 + 2 : 4;
      for (int t = seg.t0; t < seg.t1; ++t, ++g) {
        if ((g & 1) != wg) continue;
        const bool tail = t * kTile + kTile > ctx;
        // the row's view of the tile's four times 32 keys
        uint32_t see0 = 0xffffffffu, see1 = see0, see2 = see0, see3 = see0;
        if (tail) {
          see0 = sees(t * kTile);
          see1 = sees(t * kTile + 32);
          see2 = sees(t * kTile + 64);
          see3 = sees(t * kTile + 96);
        }
        auto seen = [&](int h) { return h == 0 ? see0 : h == 1 ? see1 : h == 2 ? see2 : see3; };
        w.wait(&ctl.s_full[wg], (g >> 1) & 1);
        tc_fence_after();
        // ---- a row's first reference: the maximum of its first tile with a
        // visible key
        if (__any_sync(0xffffffffu, !set)) {
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
          for (int h = h0; h < h1; ++h) {
            uint32_t u[32];
            tmem_ld32(t_s + 32 * h, u);
            tmem_ld_wait();
            if (tail) {
              const uint32_t bits = seen(h);
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if (!(bits >> c & 1u)) u[c] = 0xFF800000u;
            }
#pragma unroll
            for (int c = 0; c < 32; c += 2)
              m4[(c / 2) & 3] =
                  fmax3(m4[(c / 2) & 3], __uint_as_float(u[c]), __uint_as_float(u[c + 1]));
          }
          const float m = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * factor;
          if (!set && m > -INFINITY) {
            off = kPOffset - m;
            set = true;
          }
        }
        // ---- P, in one pass: 32 scores become 16 words over scores that were
        // read already.  A row whose 32 scores exceed its reference by more than
        // kRefLag moves it by a whole power of two, which rescales the row's
        // earlier P of this tile, its sum and O without rounding.  (But for P in
        // f16 that falls below 2^-14: it loses bits, below 2^-25 all of them.
        // Against the new maximum, which is above 2^7, that is at most 2^-32 a
        // key, far less than P's rounding at the maximum.)
        const uint64_t f2 = f2_pack(factor, factor);
#pragma unroll 1
        for (int h = h0; h < h1; ++h) {
          uint32_t u[32], p[16];
          tmem_ld32(t_s + 32 * h, u);
          tmem_ld_wait();
          if (tail) {
            const uint32_t bits = seen(h);
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (!(bits >> c & 1u)) u[c] = 0xFF800000u;
          }
          uint64_t part[2];
          float m4[4];
          auto exponentials = [&]() {
            const uint64_t o2 = f2_pack(off, off);
            part[0] = part[1] = 0;
#pragma unroll
            for (int c = 0; c < 4; ++c) m4[c] = -INFINITY;
#pragma unroll
            for (int c = 0; c < 32; c += 2) {
              float x0, x1;
              f2_unpack(f2_fma(f2_bits(u[c], u[c + 1]), f2, o2), x0, x1);
              m4[(c / 2) & 3] = fmax3(m4[(c / 2) & 3], x0, x1);
              const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
              part[(c / 2) & 1] = f2_add(part[(c / 2) & 1], f2_pack(p0, p1));
              p[c / 2] = kFp8 ? cvt_f16x2(p0, p1) : cvt_bf16x2(p0, p1);
            }
          };
          exponentials();
          const float m = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
          const bool moves = m > kPOffset + kRefLag;
          if (__any_sync(0xffffffffu, moves)) {
            const float by = moves ? floorf(kPOffset - m) : 0.0f;
            const float scale = ex2_approx(by);
            const uint64_t s2 = f2_pack(scale, scale);
            off += by;
            sum2[0] = f2_mul(sum2[0], s2);
            sum2[1] = f2_mul(sum2[1], s2);
            tmem_st_wait();
#pragma unroll 1
            for (int i = h0; i < h; ++i) {
              tmem_ld16(t_s + 16 * i, p);
              tmem_ld_wait();
#pragma unroll
              for (int c = 0; c < 16; ++c) p[c] = kFp8 ? scale_f16x2(p[c], scale) : scale_bf16x2(p[c], scale);
              tmem_st16(t_s + 16 * i, p);
            }
            // (O is complete: these scores were issued after its last product)
#pragma unroll 1
            for (int i = 0; i < 8 && g - g0 > 1; ++i) {
              tmem_ld16(t_o + 16 * i, p);
              tmem_ld_wait();
#pragma unroll
              for (int c = 0; c < 16; ++c) p[c] = __float_as_uint(__uint_as_float(p[c]) * scale);
              tmem_st16(t_o + 16 * i, p);
            }
            exponentials();
          }
          sum2[0] = f2_add(sum2[0], part[0]);
          sum2[1] = f2_add(sum2[1], part[1]);
          tmem_st16(t_s + 16 * h, p);
        }
        if (doubled) {   // the other half's keys
          uint32_t zero[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) zero[c] = 0;
          tmem_st32(t_s + 32 - 16 * h0, zero);
        }
        tmem_st_wait();
        tc_fence_before();
        w.arrive(&ctl.p_full[wg]);
      }

      // ---- epilogue: group wg takes channels 64 wg .. of a row's parts: both
      // groups', and with doubled rows the copy's
      {
        float s0, s1;
        f2_unpack(f2_add(sum2[0], sum2[1]), s0, s1);
        ctl.ml[wg][row] = make_float2(set ? kPOffset - off : -INFINITY, s0 + s1);
      }
      const int n = g - g0;
      wait_pv(g - 1);
      if (n > 1) wait_pv(g - 2);
      tc_fence_after();
      group_sync(1, C::kSoftmaxThreads);
      const bool has[2] = {n > 1 || (g0 & 1) == 0, n > 1 || (g0 & 1) == 1};
      float ref = -INFINITY, l = 0.0f, scale[2] = {0.0f, 0.0f};
      const int other = doubled ? row ^ 64 : row;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (has[i]) ref = fmaxf(ref, fmaxf(ctl.ml[i][row].x, ctl.ml[i][other].x));
      // no visible key: ref = -inf, O = 0, l = 0 (NaN scores only: l = NaN)
      auto weight = [&](float x) { return x == -INFINITY ? 1.0f : ex2_approx(x - ref); };
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (has[i]) {
          const float2 mine = ctl.ml[i][row], theirs = ctl.ml[i][other];
          scale[i] = weight(mine.x);
          l = fmaf(scale[i], mine.y, l);
          if (doubled) l = fmaf(weight(theirs.x), theirs.y, l);
        }
      const bool flagged =
          *const_cast<volatile int*>(&ctl.flagged[(unit + 1) & 3]) == unit + 1;
      const bool whole = seg.t0 == 0 && seg.t1 == seg.tiles;
      const float inv = l == 0.0f ? 0.0f : ds_v / l;
      const int out_row = rows.out_row[row];
      const int64_t piece = (2 * static_cast<int64_t>(blockIdx.x) + (seg.t0 == 0)) * R + row;
      const bool copy = doubled && row >= 64;
      const bool live = out_row >= 0 && !copy && !w.aborted();
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        const int d0 = 64 * wg + 32 * h;
        float o[32];
#pragma unroll
        for (int c = 0; c < 32; ++c) o[c] = 0.0f;
#pragma unroll 1
        for (int i = 0; i < 2; ++i)
          if (has[i]) {
            const float s = i ? scale[1] : scale[0];
            uint32_t u[32];
            tmem_ld32(tmem + lane_off + C::kO + 128 * i + d0, u);
            tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < 32; ++c) o[c] = fmaf(s, __uint_as_float(u[c]), o[c]);
          }
        if (doubled) {
          float* part = ctl.half[wg][row & 63];
          if (copy) {
#pragma unroll
            for (int c = 0; c < 32; ++c) part[c] = o[c];
          }
          group_sync(2 + wg, 128);
          if (!copy) {
#pragma unroll
            for (int c = 0; c < 32; ++c) o[c] += part[c];
          }
          group_sync(2 + wg, 128);
        }
        if (flagged) {
          for (int pos = max(ctx, seg.t0 * kTile); pos < min(seg.seq, seg.t1 * kTile); ++pos) {
            const int id = a.tables[seg.b * a.table_stride + (pos >> a.page_log2)];
            if (id < 0 || id >= a.num_pages || !(sees(pos) & 1u)) continue;
            const int64_t at = id * a.page_stride +
                               (pos & ((1 << a.page_log2) - 1)) * a.slot_stride +
                               seg.head * a.head_stride + d0;
#pragma unroll
            for (int c = 0; c < 32; ++c) o[c] += wild_value<kFp8>(a.v, at + c);
          }
        }
        if (live && whole) {
          uint4* to = reinterpret_cast<uint4*>(a.out + static_cast<int64_t>(out_row) * kHeadDim + d0);
#pragma unroll
          for (int c = 0; c < 32; c += 8) {
            uint32_t v[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const float x0 = inv == 0.0f ? 0.0f : o[c + 2 * u] * inv;
              const float x1 = inv == 0.0f ? 0.0f : o[c + 2 * u + 1] * inv;
              v[u] = cvt_bf16x2(x0, x1);
            }
            to[c / 8] = make_uint4(v[0], v[1], v[2], v[3]);
          }
        } else if (live) {
          float4* to = reinterpret_cast<float4*>(a.part_o + piece * kHeadDim + d0);
#pragma unroll
          for (int c = 0; c < 32; c += 4)
            to[c / 4] = make_float4(o[c], o[c + 1], o[c + 2], o[c + 3]);
        }
      }
      if (live && !whole && wg == 0) a.part_ml[piece] = make_float2(ref, l);
      tc_fence_before();
      group_sync(1, C::kSoftmaxThreads);   // O and `ml` may be written again
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == C::kMmaWarp) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------------
// Join: block (x, y) takes the unit that begins in CTA x's range and leaves it,
// and rows kJoinRows y .. of it, a warp per row, four channels a lane:
// out = sum_i 2^(ref_i - ref) O_i ds_v / sum_i 2^(ref_i - ref) l_i, pieces in
// order.  Bound: launch and latency; the pieces are in L2.
// ---------------------------------------------------------------------------

constexpr int kJoinThreads = 256;
constexpr int kJoinRows = 16;

template <int R, bool kFp8>
__global__ void __launch_bounds__(kJoinThreads) kv_tree_join_kernel(const TreeArgs a) {
  __shared__ float s_scale[kJoinThreads / 32][kMaxCtas];
  const float ds_v = kFp8 ? __ldg(a.descale + 2) : 1.0f;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const JoinInfo u = a.join[blockIdx.x];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i0 = warp; i0 < kJoinRows; i0 += kJoinThreads / 32) {
    const int r = blockIdx.y * kJoinRows + i0;
    const int row = u.rt * R + r;
    const int node = node_of(a, row);
    if (u.pieces == 0 || node >= u.n) return;
    // piece i; the first CTA's piece is its last one, the others' their first
    auto at = [&](int i) { return (2 * static_cast<int64_t>(blockIdx.x + i) + (i == 0)) * R + r; };
    float m = -INFINITY, l = 0.0f;
    for (int i = lane; i < u.pieces; i += 32) m = fmaxf(m, a.part_ml[at(i)].x);
#pragma unroll
    for (int off = 16; off >= 1; off /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    for (int i = lane; i < u.pieces; i += 32) {
      const float2 ml = a.part_ml[at(i)];
      // a piece of no visible key has ref = -inf, O = 0 and l = 0; one whose
      // scores were all NaN has ref = -inf and l = NaN
      const float scale = ml.x == -INFINITY ? 1.0f : exp2f(ml.x - m);
      s_scale[warp][i] = scale;
      l = fmaf(scale, ml.y, l);
    }
#pragma unroll
    for (int off = 16; off >= 1; off /= 2) l += __shfl_xor_sync(0xffffffffu, l, off);
    const float inv = l == 0.0f ? 0.0f : ds_v / l;
    __syncwarp();
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
    for (int i = 0; i < u.pieces; ++i) {
      const float s = s_scale[warp][i];
      const float4 x = *reinterpret_cast<const float4*>(a.part_o + at(i) * kHeadDim + 4 * lane);
      o.x = fmaf(s, x.x, o.x);
      o.y = fmaf(s, x.y, o.y);
      o.z = fmaf(s, x.z, o.z);
      o.w = fmaf(s, x.w, o.w);
    }
    __syncwarp();
    if (inv == 0.0f) o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const int64_t out_row = static_cast<int64_t>(u.q0 + node) * (a.kv_heads * a.group) +
                            u.head * a.group + (row - node * a.group);
    *reinterpret_cast<uint2*>(a.out + out_row * kHeadDim + 4 * lane) =
        make_uint2(cvt_bf16x2(o.x * inv, o.y * inv), cvt_bf16x2(o.z * inv, o.w * inv));
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

// Where this thread's next launch stalls its producers of K and V (self-test).
constexpr int kNoStall = -1;
thread_local int next_stall[2] = {kNoStall, kNoStall};

// Query rows of a tile.  Up to 32 rows of a KV head: keys on the lanes, with
// the fewest columns that hold them (16 is the smallest N); above: rows on the
// lanes.
int tile_rows(int max_q, int heads, int kv_heads) {
  const int64_t rows = static_cast<int64_t>(max_q) * (heads / kv_heads);
  return rows <= 16 ? 16 : rows <= 32 ? 32 : 128;
}

int launch_ctas(int rows, int max_q, int max_seqlen, int heads, int kv_heads) {
  const int64_t items = kv_tree_max_items(rows, max_q, max_seqlen, heads, kv_heads);
  const int64_t ctas = (items + kMinTreeItems - 1) / kMinTreeItems;
  return static_cast<int>(ctas < 1 ? 1 : ctas < kMaxCtas ? ctas : kMaxCtas);
}

template <int R, bool kFp8>
cudaError_t launch_t(const KvTreeLaunch& p, const TreeArgs& a, cudaStream_t stream) {
  using C = typename std::conditional<R == 128, RowsCfg<kFp8>, KeysCfg<R == 128 ? 32 : R, kFp8>>::type;
  using Control = typename std::conditional<R == 128, RowsControl<kFp8>,
                                            KeysControl<R == 128 ? 32 : R, kFp8>>::type;
  void (*kernel)(CUtensorMap, CUtensorMap, TreeArgs);
  if constexpr (R == 128) kernel = kv_tree_rows_kernel<kFp8>;
  else kernel = kv_tree_keys_kernel<R, kFp8>;
  CUtensorMap mk, mv;
  if (!make_cache_map(&mk, p.cache.k, p.cache) || !make_cache_map(&mv, p.cache.v, p.cache))
    return cudaErrorInvalidValue;
  constexpr int kSmem = 1024 + C::kSmemData + static_cast<int>(sizeof(Control));
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
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
      if (e != cudaSuccess) return e;
      attr_set |= uint64_t{1} << dev;
    }
  }
  const int ctas = launch_ctas(p.rows, p.max_q, p.max_seqlen, p.heads, p.cache.heads);
  kernel<<<ctas, C::kThreads, kSmem, stream>>>(mk, mv, a);
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
  return cudaLaunchKernelEx(&cfg, kv_tree_join_kernel<R, kFp8>, a);
}

}  // namespace

int64_t kv_tree_max_items(int rows, int max_q, int max_seqlen, int heads, int kv_heads) {
  const int R = tile_rows(max_q, heads, kv_heads);
  const int64_t tiles = (static_cast<int64_t>(max_seqlen) + kTile - 1) / kTile;
  // (each factor is below 2^31; a product beyond 2^62 counts as 2^62)
  int64_t items = (static_cast<int64_t>(max_q) * (heads / kv_heads) + R - 1) / R;
  for (int64_t f : {static_cast<int64_t>(kv_heads), static_cast<int64_t>(rows),
                    tiles > 0 ? kUnitCost + tiles : 0})
    items = f > 0 && items > (int64_t{1} << 62) / f ? int64_t{1} << 62 : items * f;
  return items;
}

size_t kv_tree_workspace_bytes(int rows, int max_q, int max_seqlen, int heads, int kv_heads) {
  const int ctas = launch_ctas(rows, max_q, max_seqlen, heads, kv_heads);
  if (ctas <= 1) return 0;
  return static_cast<size_t>(2 * ctas) * tile_rows(max_q, heads, kv_heads) *
             (kHeadDim * sizeof(float) + sizeof(float2)) +
         ctas * sizeof(JoinInfo);
}

void stall_next_kv_tree(bool v, int tile) { next_stall[v] = tile; }

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
  a.group_magic = a.group == 1 ? 0u
                               : static_cast<uint32_t>(((uint64_t{1} << 32) + a.group - 1) / a.group);
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
  a.stall_k = next_stall[0];
  a.stall_v = next_stall[1];
  next_stall[0] = next_stall[1] = kNoStall;
  const int R = tile_rows(p.max_q, p.heads, p.cache.heads);
  const int ctas = launch_ctas(p.rows, p.max_q, p.max_seqlen, p.heads, p.cache.heads);
  a.part_o = static_cast<float*>(p.workspace);
  a.part_ml = reinterpret_cast<float2*>(a.part_o + static_cast<size_t>(2 * ctas) * R * kHeadDim);
  a.join = ctas > 1 ? reinterpret_cast<JoinInfo*>(a.part_ml + static_cast<size_t>(2 * ctas) * R)
                    : nullptr;
  if (p.cache.fp8)
    return R == 16   ? launch_t<16, true>(p, a, stream)
           : R == 32 ? launch_t<32, true>(p, a, stream)
                     : launch_t<128, true>(p, a, stream);
  return R == 16   ? launch_t<16, false>(p, a, stream)
         : R == 32 ? launch_t<32, false>(p, a, stream)
                   : launch_t<128, false>(p, a, stream);
}

}  // namespace fp8attn
