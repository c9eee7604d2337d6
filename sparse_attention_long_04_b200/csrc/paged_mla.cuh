// MLA attention in MQA mode over the paged caches: single tokens (decode) and chunks of new
// tokens per sequence, over bf16 latent rows or the 8-bit rows of q8_row.cuh.
//
//   l_s = sigma * q[t,h,:] . kv[s,:],  O[t,h,:] = sum_s softmax(l)_s kv[s, 0:D_V],
//   LSE[t,h] = log sum_s exp(l_s),  s over the row's selected keys (idx) or all its keys
//
// Layout of the work: a cluster of two CTAs per query row (and split of its tiles).  O of 128
// heads x 512 values in fp32 is a whole SM's TMEM, so CTA c accumulates the value dims
// [c D_V/2, (c+1) D_V/2) of all heads.  It holds the same half of every gathered key and nothing
// else: over it it computes PARTIAL logits of all heads (the rotary dims are added by the two
// CTAs on alternate tiles), keeps those of its own 64 heads and sends the other 64 heads' to its
// partner, so that every logit is the sum of two halves.  Each CTA then runs the softmax of its
// own heads only and puts their probabilities into both CTAs' shared memory, as the A operand of
// both PV products.  Nothing is gathered, expanded, multiplied or exponentiated twice.  Per 64-key
// tile a CTA sends 16 KB of logits (st.async) and 8 KB of probabilities (a bulk copy per 32 heads)
// to its partner, counted in bytes on the receiver's barriers.
//
// Both CTAs gathering whole keys and computing all logits instead (nothing exchanged): 592 rows x
// 2048 keys of (576, 512) take 408 us from the bf16 cache and 496 us from the 8-bit one, against 362
// and 398 here.  There the shared-memory pipe is the limit (bf16 rows 98% busy: 36 KB of copies in
// and 64 + 72 KB of MMA operands a tile out).  Here no pipe is above 56%: a tile takes some 2050
// cycles because a softmax warp's chain of waits, from a tile's product to its probabilities, is
// 3500-4000 with two warps a quarter in turn, and 15% of a CTA's time is its fixed cost (indices, Q,
// filling, draining, output).  Sending the logits by bulk copies, a second logit buffer, the QK
// issuer freed of the rescaling: each as slow or slower (398 -> 411, 404, 391 with 5 slots but
// bf16 349 -> 382; measured before the fence of mbar_arrive_cluster_read, which cost bf16 rows the
// 3% between 349 and 362).
//
// Tensor work of a tile at (576, 512): 16 or 20 QK MMAs of N = 64 (32 cycles each, A in TMEM) and
// 4 PV MMAs of N = 256 (128 cycles): 1090 cycles on average.  The MMAs are issued by one elected
// lane of a converged warp (elect.sync) from precomputed descriptors: issued from an ordinary
// `lane == 0` branch with the descriptors built on the way, one costs 76-90 cycles whatever its
// size.
//
// 8-bit rows: the gather warps read the codes into registers, expand them to bf16 (exactly: the
// scales are powers of two) and store them into the same swizzled tiles the bf16 gather fills
// with cp.async; the rotary dims are bf16 in both caches and always come by cp.async.
//
// Warp roles (512 threads), q = warp % 4 being the TMEM lanes [32 q, 32 q + 32) a warp can reach
// and q / 2 the CTA that owns those heads:
//   warps 0-7 in the owner: the softmax of quarter q, warp < 4 the even tiles, the others the odd
//   warp < 4, not the owner's: q even issues the QK products, q odd the PV products, each after
//                rescaling O of its quarter when the owner moved a head's reference
//   warps 4-7, not the owner's: send quarter q's partial logits away
//   warps 8-15   resolve the keys, then gather (8 rows of every tile each)
// Without idx the keys are every prior key; a 64-key tile is then one page, and the pages of a
// split's tiles are resolved up front (kMaxDenseTiles of them).
#pragma once
#include "q8_row.cuh"
#include "rows.cuh"
#include "sm100.cuh"

namespace dsa {

struct PagedMlaParams {
  PagedSeqs s;
  const uint8_t* kv;           // cache rows: bf16 [D_QK] or Q8Row
  const int32_t* idx;          // [row_count, topk], relative to row_begin, or null
  __nv_bfloat16* out;          // [T, H, D_V]
  float* lse;                  // [T, H]
  float* part_o;               // split partials [splits, row_count, H, D_V] or null
  float* part_lse;             // [splits, row_count, H]
  int32_t row_begin, row_count, topk, h, splits;
  float scale_log2;            // sigma * log2(e)
  int32_t* status;
};

constexpr int kMaxDenseTiles = 2048;   // tiles of one split without idx
constexpr int kMaxPagedSplits = 16;    // splits of a row's tiles
// Up to this many pages a sequence (131072 keys) its block-table row is copied to shared memory, one
// coalesced trip, and the selected keys look their pages up there; looked up in global memory they
// come 1600 cycles later, since each of a warp's 8 loads touches up to 32 sectors.
constexpr int kStagedBlocks = 2048;
// Named barriers (1-4: the output's quarters).  kSetupBar: warps 0-7, behind the set-up; kGatherBar:
// warps 8-15, behind the staged table; kReadyBar: warps 8-15 wait for the set-up and for one
// another's keys; kKeysBar: warps 0-7 wait for the keys, having copied Q.
constexpr uint32_t kSetupBar = 5, kGatherBar = 6, kReadyBar = 7, kKeysBar = 8;

// Asynchronous stores into a CTA of the cluster (addr and bar are shared::cluster addresses of
// that CTA); the bytes are counted on its barrier when they have landed.
__device__ __forceinline__ void st_async_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                            uint32_t d, uint32_t bar) {
  asm volatile(
      "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, "
      "[%5];" ::"r"(addr),
      "r"(a), "r"(b), "r"(c), "r"(d), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void st_async(uint32_t addr, uint32_t a, uint32_t bar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(
                   addr),
               "r"(a), "r"(bar)
               : "memory");
}
// Copies `bytes` of this CTA's shared memory into the same cluster's CTA that `dst` and `bar` lie in,
// counted on its barrier when they have landed.
__device__ __forceinline__ void bulk_copy_cluster(uint32_t dst, uint32_t src, uint32_t bytes,
                                                  uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst), "r"(src), "r"(bytes), "r"(bar)
      : "memory");
}
// Arrive on a barrier of another CTA of the cluster when what this thread (and, behind a
// __syncwarp, its warp) read from its own CTA's shared memory has been read: the other CTA may
// overwrite it once its wait has passed.  The fence releases the accesses to this CTA's shared
// memory alone.  An arrival with release semantics of its own also waits for everything the thread
// stored elsewhere: 2048 rows over 8-bit rows 1850 us instead of 1449, 1000 rows over bf16 835
// instead of 680.
__device__ __forceinline__ void mbar_arrive_cluster_read(uint32_t bar) {
  asm volatile(
      "fence.release.sync_restrict::shared::cta.cluster;\n\t"
      "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar)
      : "memory");
}
// Arrive once on the barrier at this offset in every CTA of `mask` when every tcgen05 operation
// this thread issued so far has completed.
__device__ __forceinline__ void umma_commit_multicast(uint32_t bar, uint16_t mask) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], %1;" ::"r"(bar),
      "h"(mask)
      : "memory");
}

__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                             uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

// 2^x, results below the normal range flushed to 0 (a probability that small adds nothing).
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Tile sizes, rings and columns.
template <int D_QK, int D_V, bool kQ8>
struct PagedCfg {
  static constexpr int KB_ALL = (D_QK + 63) / 64;     // 64-dim k-blocks of a latent row
  static constexpr int V_HALF = D_V / 2;              // value dims per CTA
  static constexpr int VKB = V_HALF / 64;             // value blocks per CTA
  static constexpr int BN = 64;                       // keys per tile
  // A slot is held from QK to PV, some 3 tiles.  8-bit codes are loaded through L1, which gets what
  // shared memory leaves: with 4 slots 64 tokens over 64 contexts (rows from HBM) take 59 us, with 5
  // 66; 592 rows of one context (rows from L2) 398 and 392.  cp.async rows pass L1 by: 357 and 349.
  static constexpr int V_SLOTS = kQ8 ? 4 : 5;
  static constexpr int MAX_TILES = 32;                // topk <= 2048
  static constexpr int THREADS = 512;
  static constexpr int GATHER = 256;                  // gathering threads
  // TMEM: O, S, the rotary block of Q, the CTA's value blocks of Q
  static constexpr int S_COL = V_HALF;
  static constexpr int QR_COL = S_COL + BN;
  static constexpr int Q_COL = QR_COL + 32;
  static constexpr int TMEM_USED = Q_COL + VKB * 32;
  static constexpr int TMEM_COLS = TMEM_USED <= 256 ? 256 : 512;
  static constexpr int KB_BYTES = BN * 128;           // one k-block of a tile
  static constexpr int V_SLOT_BYTES = VKB * KB_BYTES;
  static constexpr int Q_KB_BYTES = 128 * 128;        // one k-block of Q
  static constexpr int P_BYTES = 128 * 128;           // 128 heads x 64 keys bf16, twice
  static constexpr int X_BYTES = BN * 64 * 4;         // partial logits of 64 heads
  static constexpr int P_TX = 64 * 128 + 64 * 4;      // the partner's probabilities and rescales
  // (the dynamic array starts on a 1024-byte boundary: the kernel has no static shared memory)
  static constexpr int BARS = 39;
  static constexpr int SMEM_USED = V_SLOTS * V_SLOT_BYTES + KB_BYTES + 2 * P_BYTES + X_BYTES +
                                   MAX_TILES * BN * 4 + MAX_TILES * 12 + 8 * 64 * 4 + BARS * 8;
  // at least 116 KB, so that one CTA runs per SM (its TMEM allocation never waits)
  static constexpr int SMEM_BYTES = SMEM_USED > 116 * 1024 ? SMEM_USED : 116 * 1024;
  static_assert(V_HALF % 64 == 0 && V_HALF <= 256, "PV MMA N");
  static_assert(2 * VKB + 1 == KB_ALL, "value blocks and one rotary block");
  static_assert(TMEM_USED <= 512, "TMEM columns");
  static constexpr int Q_OFF = V_SLOTS * V_SLOT_BYTES - (VKB + 1) * Q_KB_BYTES;   // Q staging
  static constexpr int PRE_TILES = Q_OFF / V_SLOT_BYTES;      // slots in front of it
  static_assert(Q_OFF >= 0, "Q staging fits the ring");
  static_assert(128 * (V_HALF * 4 + 16) <= V_SLOTS * V_SLOT_BYTES + KB_BYTES,
                "output staging fits the ring and the rotary block behind it");
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
};

// Multiplies COLS columns of O (this warp's lanes) by alpha.
template <int COLS>
__device__ __forceinline__ void rescale_o(uint32_t addr, float alpha) {
#pragma unroll 1
  for (int c0 = 0; c0 < COLS; c0 += 32) {
    uint32_t u[32];
    tmem_ld32(addr + c0, u);
    tmem_wait_ld();
#pragma unroll
    for (int j = 0; j < 32; ++j) u[j] = __float_as_uint(__uint_as_float(u[j]) * alpha);
    tmem_st32(addr + c0, u);
  }
  tmem_wait_st();
}

// Grid: x = 2 * row + c (clusters of two), y = split.
template <int D_QK, int D_V, bool kQ8>
__global__ void __launch_bounds__(512, 1)
    dsa_paged_mla_kernel(const __grid_constant__ CUtensorMap q_map, const PagedMlaParams p) {
  using C = PagedCfg<D_QK, D_V, kQ8>;
  using R = Q8Row<D_QK, D_V>;
  constexpr int ROW_BYTES = kQ8 ? R::BYTES : D_QK * 2;
  static_assert(R::ROPE <= 64 && D_V % 128 == 0, "rotary dims fill (part of) the last k-block");
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sV = smem;                                           // [V_SLOTS]
  uint8_t* sQ = sV + C::Q_OFF;                                  // Q, before the ring needs it
  uint8_t* sR = sV + C::V_SLOTS * C::V_SLOT_BYTES;              // rotary block of a tile
  uint8_t* sP = sR + C::KB_BYTES;                               // [2] probabilities, all heads
  uint8_t* sX = sP + 2 * C::P_BYTES;   // [16 key quads][64 heads][4]: the partner's half logits
  // selected: the physical row of every key; dense: the first physical row of every tile
  int32_t* sPhys = reinterpret_cast<int32_t*>(sX + C::X_BYTES);                   // [2048]
  uint64_t* sMask = reinterpret_cast<uint64_t*>(sPhys + C::MAX_TILES * C::BN);   // [32]
  int32_t* sTiles = reinterpret_cast<int32_t*>(sMask + C::MAX_TILES);            // [32]
  float* sAlpha = reinterpret_cast<float*>(sTiles + C::MAX_TILES);   // [2][64] from the partner
  float* sRef = sAlpha + 2 * 64;                  // [2][64 heads] the reference after a tile
  float* sSum = sRef + 2 * 64;                    // [2 warps][sum, reference][64 heads]
  uint64_t* bars = reinterpret_cast<uint64_t*>(sSum + 4 * 64);
  // [128] 1 / sum, half of it written by the partner after its last tile.  Nothing before the tiles
  // touches this memory, and the factors in it have been read in front of the last PV, which the
  // partner's softmax warps wait for.  (Over the key rows, a CTA without a tile could still be
  // storing them when its partner writes; sSum too: with one tile a softmax warp has none and
  // writes its sums at once.)
  float* sInv = sAlpha;
  uint64_t* v_full = bars;           // [V_SLOTS] every gathering thread
  uint64_t* v_empty = bars + 5;      // [V_SLOTS] PV commit
  uint64_t* r_full = bars + 10;      // every gathering thread (rotary copies landed)
  uint64_t* r_empty = bars + 11;     // QK commit of a rotary tile
  uint64_t* s_full = bars + 12;      // [2 tiles] QK commit
  uint64_t* s_empty = bars + 14;     // the 2 softmax warps of the tile and the 2 senders
  uint64_t* x_full = bars + 15;      // [2 tiles][2 key halves] a local arrival + the partner's bytes
  uint64_t* x_free = bars + 19;      // [2 key halves] the partner's 2 softmax warps have read it
  uint64_t* p_full = bars + 21;      // [2] 2 local softmax warps + P_TX bytes from the partner
  uint64_t* p_empty = bars + 23;     // [2] both CTAs' PV commits
  uint64_t* o_ok = bars + 25;        // [2] the QK issuer has rescaled its quarter of O
  uint64_t* pv_done = bars + 27;     // [2] PV commit
  uint64_t* m_full = bars + 29;      // [2 quarters][2] the reference after a tile is in sRef
  uint64_t* mma_fin = bars + 33;     // [2] every MMA of an issuer completed
  uint64_t* q_bar = bars + 35;       // 1 arrival + Q bytes
  volatile uint32_t& tmem_base_s = *reinterpret_cast<volatile uint32_t*>(bars + 36);
  volatile int& abort_s = *reinterpret_cast<volatile int*>(bars + 37);
  volatile int& n_act_s = *reinterpret_cast<volatile int*>(bars + 38);
  static_assert(kMaxDenseTiles <= C::MAX_TILES * C::BN, "dense tiles fit the key array");

  wait_prior_grid();   // (launched early: the indices come from the previous kernel)
  if (p.part_o != nullptr) allow_next_grid();   // the combining kernel
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int c = static_cast<int>(cluster_ctarank());   // value half, and the heads it owns
  const uint32_t peer = static_cast<uint32_t>(c ^ 1);
  const int split = blockIdx.y;
  const int r = blockIdx.x >> 1;
  const int row = p.row_begin + r;
  const bool dense = p.idx == nullptr;
  const int n_tiles_all = p.topk / C::BN;

  // ---- the selected keys' indices, loaded first: warp 8 + pw resolves tiles pw, pw + 8, ...
  constexpr int TPW = C::MAX_TILES / 8;
  int v[2 * TPW];
  if (warp >= 8 && !dense) {
    const int32_t* irow = p.idx + static_cast<int64_t>(r) * p.topk + lane;
#pragma unroll
    for (int j = 0; j < TPW; ++j) {
      const int tt = warp - 8 + 8 * j;
      v[2 * j] = tt < n_tiles_all ? irow[tt * C::BN] : -1;
      v[2 * j + 1] = tt < n_tiles_all ? irow[tt * C::BN + 32] : -1;
    }
  }
  // ---- set-up, under those loads
  if (threadIdx.x == 0) {
    // Q: the rotary block and the CTA's value blocks into the end of the (still idle) ring, h rows a
    // block (lanes past h hold whatever was there and are never written out)
    mbar_init(smem_u32(q_bar), 1);
    fence_mbar_init();
    const uint32_t kb_bytes = static_cast<uint32_t>(p.h) * 128u;
    tma_prefetch_desc(&q_map);
    mbar_arrive_expect_tx(smem_u32(q_bar), (C::VKB + 1) * kb_bytes);
    for (int j = 0; j <= C::VKB; ++j)
      tma_load_2d(smem_u32(sQ + j * C::Q_KB_BYTES), &q_map, smem_u32(q_bar),
                  (j == 0 ? C::KB_ALL - 1 : c * C::VKB + j - 1) * 128, r * p.h);
  }
  if (warp == 1) tmem_alloc(smem_u32(bars + 36), C::TMEM_COLS);
  if (warp == 2) {
    for (int i = lane; i < 35; i += 32) {
      const uint64_t* bar = bars + i;
      const bool gather = bar < v_empty || bar == r_full;
      const bool pairs = bar >= x_free && bar < o_ok;       // x_free, p_full, p_empty
      mbar_init(smem_u32(bar), gather ? C::GATHER : bar == s_empty ? 4 : pairs ? 2 : 1);
    }
    fence_mbar_init();
    if (lane == 0) abort_s = 0;
  }
  bool bad_idx = false;
  if (warp < 8) {
    named_bar_sync(kSetupBar, 256);
    named_bar_arrive(kReadyBar, 512);
    if (warp >= 4) {
      // ---- Q from the staging area into TMEM: head = lane, two dims a column
      const int hrow = (warp & 3) * 32 + lane;
      const uint32_t lane_addr = tmem_base_s + (static_cast<uint32_t>((warp & 3) * 32) << 16);
      if (!(warp_wait(smem_u32(q_bar), 0))) {
        abort_s = 1;
        if (p.status) atomicOr(p.status, kStatusTimeout);
      } else {
        for (int kb = 0; kb <= C::VKB; ++kb) {
          uint32_t u[32];
          const uint8_t* src = sQ + kb * C::Q_KB_BYTES;
#pragma unroll
          for (int ch = 0; ch < 8; ++ch) {
            const uint4 q4 = *reinterpret_cast<const uint4*>(src + sw128_offset(hrow, ch));
            u[4 * ch + 0] = q4.x;
            u[4 * ch + 1] = q4.y;
            u[4 * ch + 2] = q4.z;
            u[4 * ch + 3] = q4.w;
          }
          tmem_st32(lane_addr + C::QR_COL + kb * 32, u);
        }
        tmem_wait_st();
      }
    }
    // Behind the cluster barrier the staging area is free for the ring and both CTAs' barriers are
    // ready.  It is arrived at early (a releasing arrival waits some 2000 cycles for the warp's memory
    // operations); the gathering warps fill the first PRE_TILES slots, which the staging area
    // leaves free, before they wait for it.
    tc_fence_before();
    __syncwarp();
    cluster_arrive();
    named_bar_sync(kKeysBar, 512);
  } else {
    cluster_arrive_relaxed();
    int b, pos;
    bool bad_row;
    paged_row(p.s, row, &b, &pos, &bad_row);
    const int n_keys = max(pos + 1, 0);
    if (bad_row && threadIdx.x == 256 && p.status) atomicOr(p.status, kStatusBadIndex);
    if (!dense) {
      // ---- every selected key -> physical row (or -1); per tile the valid-key mask; invalid keys
      // borrow the tile's first valid row
      int32_t* sTable = reinterpret_cast<int32_t*>(sP);     // (P comes later)
      const int blocks = (p.s.max_seqlen + 63) / 64;
      const bool staged = p.s.block_table != nullptr && blocks <= kStagedBlocks;
      if (staged) {
        const int32_t* table = p.s.block_table + static_cast<int64_t>(b) * p.s.max_blocks;
        const int e0 = static_cast<int>(threadIdx.x) - 256;
        int32_t t[kStagedBlocks / 256];
#pragma unroll
        for (int j = 0; j < kStagedBlocks / 256; ++j)
          t[j] = e0 + 256 * j < blocks ? __ldg(table + e0 + 256 * j) : -1;
#pragma unroll
        for (int j = 0; j < kStagedBlocks / 256; ++j)
          if (e0 + 256 * j < blocks) sTable[e0 + 256 * j] = t[j];
        named_bar_sync(kGatherBar, 256);
      }
      int32_t phys[2 * TPW];
      if (staged) {                               // (no branches: all lookups at once)
#pragma unroll
        for (int j = 0; j < 2 * TPW; ++j) {
          const bool in = v[j] >= 0 && v[j] < n_keys;
          const int64_t at = static_cast<int64_t>(sTable[in ? v[j] >> 6 : 0]) * 64 + (v[j] & 63);
          phys[j] = in && at >= 0 && at < p.s.num_kv_rows ? static_cast<int32_t>(at) : -1;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 2 * TPW; ++j)
          phys[j] = v[j] >= 0 && v[j] < n_keys
                        ? static_cast<int32_t>(paged_phys(p.s, b, v[j])) : -1;
      }
#pragma unroll
      for (int j = 0; j < 2 * TPW; ++j) bad_idx |= v[j] >= 0 && phys[j] < 0;
#pragma unroll
      for (int j = 0; j < TPW; ++j) {
        const int tt = warp - 8 + 8 * j;
        const uint32_t lo = __ballot_sync(0xffffffffu, phys[2 * j] >= 0);
        const uint32_t hi = __ballot_sync(0xffffffffu, phys[2 * j + 1] >= 0);
        const int32_t first = __shfl_sync(0xffffffffu, lo != 0 ? phys[2 * j] : phys[2 * j + 1],
                                          max(__ffs(lo != 0 ? lo : hi) - 1, 0));
        if (tt < n_tiles_all) {
          sPhys[tt * C::BN + lane] = phys[2 * j] >= 0 ? phys[2 * j] : first;
          sPhys[tt * C::BN + 32 + lane] = phys[2 * j + 1] >= 0 ? phys[2 * j + 1] : first;
          if (lane == 0) sMask[tt] = (static_cast<uint64_t>(hi) << 32) | lo;
        }
      }
    }
    if (dense && warp == 8) {
      // ---- this split's tiles (one page each) whose page is inside the cache, in key order;
      // only the row's last tile can be partial
      const int tiles = (n_keys + C::BN - 1) / C::BN;
      const int per = (tiles + p.splits - 1) / p.splits;
      const int t0 = min(tiles, split * per);
      const int t1 = min(tiles, t0 + min(per, kMaxDenseTiles));
      int cnt = 0;
      bool tail = false;
      for (int base = t0; base < t1; base += 32) {
        const int t = base + lane;
        int64_t ph = -1;
        if (t < t1) {
          ph = paged_phys(p.s, b, t * C::BN);
          // every key of the tile that the row sees must be inside the cache
          const int n = min(C::BN, n_keys - t * C::BN);
          if (ph >= 0 && ph + n > p.s.num_kv_rows) ph = -1;
          bad_idx |= ph < 0;
        }
        const uint32_t good = __ballot_sync(0xffffffffu, ph >= 0);
        if (ph >= 0) sPhys[cnt + __popc(good & ((1u << lane) - 1u))] = static_cast<int32_t>(ph);
        cnt += __popc(good);
        const int last = tiles - 1 - base;
        if (last >= 0 && last < 32) tail = (good >> last) & 1u;
      }
      if (lane == 0) {
        n_act_s = cnt;
        const int rem = n_keys - (tiles - 1) * C::BN;    // keys of the row's last tile
        // sMask[0]: the mask of the last active tile
        sMask[0] = tail && rem < C::BN ? (1ull << rem) - 1ull : ~0ull;
      }
    }
    if (bad_idx && p.status) atomicOr(p.status, kStatusBadIndex);
    named_bar_sync(kReadyBar, 512);
    named_bar_arrive(kKeysBar, 512);
  }
  // ---- the active tiles of this split, identical in both CTAs of the row (every warp writes the
  // same list, to read it without another barrier)
  int n_act;
  if (dense) {
    n_act = n_act_s;
  } else {
    const bool active = lane < n_tiles_all && sMask[lane] != 0;
    const uint32_t act = __ballot_sync(0xffffffffu, active);
    const int cnt = __popc(act), at = __popc(act & ((1u << lane) - 1u));
    const int per = (cnt + p.splits - 1) / p.splits;
    const int t0 = min(cnt, split * per);
    const int t1 = min(cnt, t0 + per);
    if (active && at >= t0 && at < t1) sTiles[at - t0] = lane;
    n_act = t1 - t0;
    __syncwarp();
  }
  if (warp < 8) cluster_wait();
  tc_fence_after();
  const uint32_t tmem = tmem_base_s;
  // (one answer for a warp's lanes, whenever another warp gives up)
  auto aborted = [&] { return __any_sync(0xffffffffu, abort_s) != 0; };
  const int n = warp < 8 && aborted() ? 0 : n_act;
  auto mask_of = [&](int i) -> uint64_t {
    if (dense) return i == n - 1 ? sMask[0] : ~0ull;
    return sMask[sTiles[i]];
  };
  // physical row of key rr of active tile i (keys past a dense row borrow the tile's first)
  auto phys_of = [&](int i, int rr) -> int64_t {
    if (!dense) return sPhys[sTiles[i] * C::BN + rr];
    const int64_t base = sPhys[i];
    return ((mask_of(i) >> rr) & 1ull) ? base + rr : base;
  };

  const int q = warp & 3;                          // TMEM lane quarter of this warp
  const bool own = (q >> 1) == c;                  // whose heads this CTA owns
  // O of a quarter the partner owns, to the references of tile j (this warp's lanes)
  auto fix_o = [&](int j) -> bool {
    const float alpha = sAlpha[(j & 1) * 64 + (q & 1) * 32 + lane];
    if (j < 1 || !__any_sync(0xffffffffu, alpha != 1.f)) return true;
    if (!warp_wait(smem_u32(&pv_done[(j - 1) & 1]), ((j - 1) >> 1) & 1)) return false;
    tc_fence_after();
    rescale_o<C::V_HALF>(tmem + (static_cast<uint32_t>(q * 32) << 16), alpha);
    tc_fence_before();
    return true;
  };
  if (warp < 4 && !own && (q & 1) == 0) {
    // ------------------------------------------------------------ QK issuer
    constexpr uint32_t idesc = idesc_f32acc(1 /* bf16 */, 128, C::BN, 0, 0);
    const uint64_t rd = sdesc_sw128(smem_u32(sR), 16, 1024);
    const uint32_t d = tmem + C::S_COL;
    bool ok = true;
    int vs = 0;
    uint32_t vph = 0;
#pragma unroll 1
    for (int i = 0; i < n + 2 && ok; ++i) {
      if (i < n) {
        const bool rot = (i & 1) == c;               // this CTA adds the tile's rotary dims
        const uint64_t vd = sdesc_sw128(smem_u32(sV + vs * C::V_SLOT_BYTES), 16, 1024);
        ok = warp_wait(smem_u32(&v_full[vs]), vph) &&
             (!rot || warp_wait(smem_u32(r_full), (i >> 1) & 1)) &&
             (i < 1 || warp_wait(smem_u32(s_empty), (i - 1) & 1));
        if (!ok) break;
        tc_fence_after();
        fence_proxy_async_smem();   // the rows were written by cp.async and ordinary stores
        if (elect_one()) {
          if (rot) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma_bf16_ts(d, tmem + C::QR_COL + k * 8, rd + k * 2, idesc, k != 0);
            umma_commit(smem_u32(r_empty));
          }
#pragma unroll
          for (int k = 0; k < 4 * C::VKB; ++k)
            umma_bf16_ts(d, tmem + C::Q_COL + k * 8,
                         vd + ((k / 4) * C::KB_BYTES + (k % 4) * 32) / 16, idesc, rot || k != 0);
          umma_commit(smem_u32(&s_full[i & 1]));
        }
        __syncwarp();
        if (++vs == C::V_SLOTS) {
          vs = 0;
          vph ^= 1u;
        }
      }
      if (i >= 2) {                                  // O of this quarter for PV(i - 2)
        const int j = i - 2;
        ok = warp_wait<true>(smem_u32(&p_full[j & 1]), (j >> 1) & 1) && fix_o(j);
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(smem_u32(&o_ok[j & 1]));
      }
    }
    if (!ok) {
      abort_s = 1;
      if (lane == 0 && p.status) atomicOr(p.status, kStatusTimeout);
    }
    __syncwarp();
    if (elect_one()) umma_commit(smem_u32(&mma_fin[0]));   // no MMA may outlive the CTA
    __syncwarp();
    warp_wait(smem_u32(&mma_fin[0]), 0);
  } else if (warp < 4 && !own) {
    // ------------------------------------------------------------ PV issuer
    constexpr uint32_t idesc = idesc_f32acc(1, 128, C::V_HALF, 0, 1);
    bool ok = true;
    int vs = 0;
#pragma unroll 1
    for (int j = 0; j < n && ok; ++j) {
      const int b2 = j & 1;
      const uint64_t vd = sdesc_sw128(smem_u32(sV + vs * C::V_SLOT_BYTES), C::KB_BYTES, 1024);
      const uint64_t pd = sdesc_sw128(smem_u32(sP + b2 * C::P_BYTES), 16, 1024);
      ok = warp_wait<true>(smem_u32(&p_full[b2]), (j >> 1) & 1) && fix_o(j) &&
           warp_wait(smem_u32(&o_ok[b2]), (j >> 1) & 1);
      if (!ok) break;
      tc_fence_after();
      fence_proxy_async_smem();   // P was written by ordinary stores and by the partner's copy
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < C::BN / 16; ++k)
          umma_bf16(tmem, pd + k * 2, vd + k * 16 * 128 / 16, idesc, j > 0 || k != 0);
        umma_commit(smem_u32(&v_empty[vs]));
        umma_commit(smem_u32(&pv_done[b2]));
        umma_commit_multicast(smem_u32(&p_empty[b2]), 3);
      }
      __syncwarp();
      if (++vs == C::V_SLOTS) vs = 0;
    }
    if (!ok) {
      abort_s = 1;
      if (lane == 0 && p.status) atomicOr(p.status, kStatusTimeout);
    }
    __syncwarp();
    if (elect_one()) umma_commit(smem_u32(&mma_fin[1]));
    __syncwarp();
    warp_wait(smem_u32(&mma_fin[1]), 0);
  } else if (warp >= 8) {
    // ------------------------------------------------------------ gather
    // warp 8 + pw fills rows [8 pw, 8 pw + 8) of each tile
    const int pw = warp - 8;
    const int ch = lane & 7;                    // 16-byte chunk of a 128-byte row block
    const int rsub = lane >> 3;                 // rows rsub, rsub + 4
    const int kb0 = c * C::VKB;                 // the CTA's first latent block
    // Physical rows, one tile ahead: lane l holds that of row 8 pw + l % 8, the others come by
    // shuffle, so that no copy waits for a chain of shared-memory loads.
    auto rows_of = [&](int i) { return static_cast<int32_t>(phys_of(i, pw * 8 + (lane & 7))); };
    auto row_ptr = [&](int32_t rows, int l) {
      return p.kv + static_cast<int64_t>(__shfl_sync(0xffffffffu, rows, l)) * ROW_BYTES;
    };
    // a block of bf16 rows straight from the cache, its chunks past `valid` zeros
    auto copy_block = [&](uint8_t* dst, const uint8_t* const (&src)[2], int byte, int valid) {
      const bool in = ch < valid;
#pragma unroll
      for (int j = 0; j < 2; ++j)
        cp_async_16(smem_u32(dst) + sw128_offset(pw * 8 + rsub + 4 * j, ch),
                    in ? src[j] + byte + ch * 16 : p.kv, in ? 16u : 0u);
    };
    // 8-bit codes: lane = 16-code chunk lane % 4 of row lane / 4, every value block of the CTA.  Eight
    // lanes, two neighbouring rows, then store to the eight different 16-byte columns of a swizzled
    // tile (eight lanes on one row would meet two to a column: 8.1 instead of 4 wavefronts a
    // store).  Two register sets take turns: the set just stored is loaded with the codes and
    // scales of two tiles on, so that their latency goes by under a whole tile.
    constexpr int GP = (C::VKB + 1) / 2;         // scales of a row's half (128 values, 2 blocks)
    struct CodeSet {
      uint4 code[C::VKB];
      float scale[GP];
    };
    const int cl = lane & 3, rl = pw * 8 + (lane >> 2);
    auto load_set = [&](CodeSet& x, int32_t rows) {
      const uint8_t* src = row_ptr(rows, lane >> 2);
#pragma unroll
      for (int g = 0; g < GP; ++g)
        x.scale[g] = __ldg(reinterpret_cast<const float*>(src + R::SCALE_OFF) + kb0 / 2 + g);
#pragma unroll
      for (int ks = 0; ks < C::VKB; ++ks)
        x.code[ks] = __ldg(reinterpret_cast<const uint4*>(src + (kb0 + ks) * 64) + cl);
    };
    auto store_set = [&](const CodeSet& x, uint8_t* dst) {
#pragma unroll
      for (int ks = 0; ks < C::VKB; ++ks) {
        uint8_t* at = dst + ks * C::KB_BYTES;
        *reinterpret_cast<uint4*>(at + sw128_offset(rl, 2 * cl)) =
            q8_expand8(make_uint2(x.code[ks].x, x.code[ks].y), x.scale[ks / 2]);
        *reinterpret_cast<uint4*>(at + sw128_offset(rl, 2 * cl + 1)) =
            q8_expand8(make_uint2(x.code[ks].z, x.code[ks].w), x.scale[ks / 2]);
      }
    };
    bool ok = true, joined = false;
    int vs = 0;
    uint32_t vph = 1;                            // (the first use of each slot does not wait)
    // tile i (physical rows `rows`): its slots waited for, filled, and the barriers told; the set x
    // is then loaded with tile i + 2 (rows `rows2`)
    auto fill = [&](CodeSet& x, int i, int32_t rows, int32_t rows2) -> bool {
      if (i == C::PRE_TILES) {                   // from here on the slots were Q's staging area
        cluster_wait();
        joined = true;
        if (aborted()) return false;
      }
      const uint8_t* const src[2] = {row_ptr(rows, rsub), row_ptr(rows, rsub + 4)};
      if ((i & 1) == c) {                        // the rotary block, on this CTA's tiles
        if (i >= 2 && !warp_wait(smem_u32(r_empty), ((i >> 1) - 1) & 1)) return false;
        copy_block(sR, src, kQ8 ? R::ROPE_OFF : 2 * D_V, R::ROPE / 8);
        cp_async_arrive_noinc(smem_u32(r_full));
      }
      if (i >= C::V_SLOTS && !warp_wait(smem_u32(&v_empty[vs]), vph)) return false;
      uint8_t* dst = sV + vs * C::V_SLOT_BYTES;
      uint64_t* full = &v_full[vs];
      if (++vs == C::V_SLOTS) {
        vs = 0;
        vph ^= 1u;
      }
      if constexpr (kQ8) {
        store_set(x, dst);
        fence_proxy_async_smem();              // this thread's stores, before the MMAs read them
        mbar_arrive(smem_u32(full));
        if (i + 2 < n) load_set(x, rows2);
      } else {
#pragma unroll
        for (int ks = 0; ks < C::VKB; ++ks)
          copy_block(dst + ks * C::KB_BYTES, src, (kb0 + ks) * 128, 8);
        cp_async_arrive_noinc(smem_u32(full));
      }
      return true;
    };
    CodeSet set0, set1;
    int32_t rows0 = n > 0 ? rows_of(0) : 0, rows1 = n > 1 ? rows_of(1) : 0;
    if constexpr (kQ8) {
      if (n > 0) load_set(set0, rows0);
      if (n > 1) load_set(set1, rows1);
    }
#pragma unroll 1
    for (int i = 0; i < n && ok; i += 2) {       // (the sets by name: a copy would wait for its loads)
      const int32_t rows2 = i + 2 < n ? rows_of(i + 2) : 0, rows3 = i + 3 < n ? rows_of(i + 3) : 0;
      ok = fill(set0, i, rows0, rows2);
      if (ok && i + 1 < n) ok = fill(set1, i + 1, rows1, rows3);
      rows0 = rows2;
      rows1 = rows3;
    }
    if (!ok) {
      abort_s = 1;
      if (p.status) atomicOr(p.status, kStatusTimeout);
    }
    if (!joined) cluster_wait();
    cp_async_wait_all();   // nothing may still be writing this CTA's shared memory at exit
  } else if (!own) {
    // ------------------------------------------------------------ partial logits to their owner
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(q * 32) << 16) + C::S_COL;
    const uint32_t dst = map_to_rank(smem_u32(sX), peer) + ((q & 1) * 32 + lane) * 16;
    const uint32_t bar = map_to_rank(smem_u32(x_full), peer);
    bool ok = true;
#pragma unroll 1
    for (int i = 0; i < n && ok; ++i) {
      ok = warp_wait(smem_u32(&s_full[i & 1]), (i >> 1) & 1);
      if (!ok) break;
      tc_fence_after();
      uint32_t su[2][32];
      tmem_ld32(lane_addr, su[0]);
      tmem_ld32(lane_addr + 32, su[1]);
      tmem_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(s_empty));
#pragma unroll
      for (int h = 0; h < 2; ++h) {               // 32 keys at a time
        // (the partner has read this half of the tile before)
        if (ok && i >= 1) ok = warp_wait<true>(smem_u32(&x_free[h]), (i - 1) & 1);
        if (!ok) break;
#pragma unroll
        for (int g = 0; g < 8; ++g)
          st_async_v4(dst + (h * 8 + g) * (64 * 16), su[h][4 * g], su[h][4 * g + 1],
                      su[h][4 * g + 2], su[h][4 * g + 3], bar + (2 * (i & 1) + h) * 8);
      }
    }
    // (every arrival that the partner owes has landed before the CTA can leave)
    for (int h = 0; h < 2 && ok && n > 0; ++h)
      ok = warp_wait<true>(smem_u32(&x_free[h]), (n - 1) & 1);
    if (!ok) {
      abort_s = 1;
      if (lane == 0 && p.status) atomicOr(p.status, kStatusTimeout);
    }
  } else {
    // ------------------------------------------------------------ softmax of the CTA's heads
    // Two warps a quarter take turns tile by tile; each hands the other the heads' references.
    const int t = warp >> 2;
    const int hrow = q * 32 + lane;             // head = TMEM lane
    const int hloc = hrow & 63;
    const bool head = hrow < p.h;               // (small shapes: MMA rows past the heads)
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(q * 32) << 16);
    const float4* xin = reinterpret_cast<const float4*>(sX) + hloc;
    const uint32_t x_free_peer = map_to_rank(smem_u32(x_free), peer);
    const uint32_t p_peer = map_to_rank(smem_u32(sP), peer) + t * C::P_BYTES + q * 32 * 128;
    const uint32_t alpha_peer = map_to_rank(smem_u32(sAlpha + t * 64 + hloc), peer);
    const uint32_t p_full_peer = map_to_rank(smem_u32(&p_full[t]), peer);
    // (16-byte chunk g of the head's row lies at XOR 16 g)
    const uint32_t p_own = smem_u32(sP) + t * C::P_BYTES + sw128_offset(hrow, 0);
    const uint32_t p_rows = smem_u32(sP) + t * C::P_BYTES + q * 32 * 128;
    const uint32_t xb = smem_u32(&x_full[2 * t]);
    const bool counts = (q & 1) == 0;           // one of the tile's two warps expects the bytes
    const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
    float m_mine = -INFINITY, l_sum = 0.f;      // l_sum: this warp's tiles, to reference m_mine
    bool ok = !aborted();
#pragma unroll 1
    for (int i = t; i < n && ok; i += 2) {
      const uint32_t ph = (i >> 1) & 1;
      if (counts && lane == 0) {
        mbar_arrive_expect_tx(xb, C::X_BYTES / 2);
        mbar_arrive_expect_tx(xb + 8, C::X_BYTES / 2);
      }
      ok = warp_wait(smem_u32(&s_full[t]), ph);
      if (!ok) break;
      tc_fence_after();
      float2 s[32];                               // the logits of 64 keys, two to a register pair
      {
        uint32_t su[2][32];
        tmem_ld32(lane_addr + C::S_COL, su[0]);
        tmem_ld32(lane_addr + C::S_COL + 32, su[1]);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e)
          s[e] = make_float2(__uint_as_float(su[e / 16][2 * (e % 16)]),
                             __uint_as_float(su[e / 16][2 * (e % 16) + 1]));
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(s_empty));
      // (the waits that this tile's probabilities need are passed where the warp waits for the
      // partner anyway: the other warp's references here, the P buffer between the key halves, when
      // the partner may already send the next tile's first half.  Behind the maxima: 592 rows in
      // 396 instead of 391 us from 8-bit rows, 362 instead of 349 from bf16.)
      float m_old = -INFINITY;
      if (i >= 1) {
        ok = warp_wait(smem_u32(&m_full[(q & 1) * 2 + (t ^ 1)]), ((i - 1) >> 1) & 1);
        if (!ok) break;
        m_old = sRef[(t ^ 1) * 64 + hloc];
      }
      // ---- plus the partner's half of these logits, 32 keys at a time
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h == 1 && ok && i >= 2)                 // both PV(i - 2)
          ok = warp_wait<true>(smem_u32(&p_empty[t]), ph ^ 1u);
        if (ok) ok = warp_wait<true>(xb + h * 8, ph);
        if (!ok) break;
#pragma unroll
        for (int g = 8 * h; g < 8 * h + 8; ++g) {
          const float4 x = xin[g * 64];
          s[2 * g] = __fadd2_rn(s[2 * g], make_float2(x.x, x.y));
          s[2 * g + 1] = __fadd2_rn(s[2 * g + 1], make_float2(x.z, x.w));
        }
        __syncwarp();                               // every lane has read its logits
        if (lane == 0) mbar_arrive_cluster_read(x_free_peer + h * 8);
      }
      if (!ok) break;
      if (mask_of(i) != ~0ull) {                  // invalid keys: -inf, so p = 0
        const uint64_t vmask = mask_of(i);
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          if (!((vmask >> (2 * e)) & 1u)) s[e].x = -INFINITY;
          if (!((vmask >> (2 * e + 1)) & 1u)) s[e].y = -INFINITY;
        }
      }
      // ---- the heads' references: moved only when a tile beats them by 2^8 (p and the sums stay far
      // inside fp32 and bf16 either way), handed on to the other warp before the exponentials
      float mm[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) mm[e] = fmaxf(s[e].x, s[e].y);
#pragma unroll
      for (int e = 4; e < 32; ++e) mm[e & 3] = fmaxf(fmaxf(mm[e & 3], s[e].x), s[e].y);
      const float m_tile = fmaxf(fmaxf(mm[0], mm[1]), fmaxf(mm[2], mm[3])) * p.scale_log2;
      const float m_ref = head && m_tile > m_old + 8.0f ? m_tile : m_old;
      sRef[t * 64 + hloc] = m_ref;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&m_full[(q & 1) * 2 + t]));
      // ---- p = 2^(sigma log2e s - reference) into shared memory, two keys to an instruction.  The
      // denominator sums the fp32 probabilities, only the PV operand is rounded (bf16: the MMA's
      // operand type).
      float2 rs[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      const float nm = m_ref != -INFINITY ? -m_ref : 0.f;   // (-inf logits only: p = 0, not NaN)
      const float2 nm2 = make_float2(nm, nm);
#pragma unroll
      for (int g = 0; g < 8; ++g) {               // 8 keys: a 16-byte chunk of P
        uint32_t pk[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 x = __ffma2_rn(s[4 * g + e], sc2, nm2);
          const float2 pr = make_float2(exp2_approx(x.x), exp2_approx(x.y));
          rs[e & 1] = __fadd2_rn(rs[e & 1], pr);
          const __nv_bfloat162 two = __float22bfloat162_rn(pr);
          pk[e] = *reinterpret_cast<const uint32_t*>(&two);
        }
        st_shared_v4(p_own ^ (g * 16), pk[0], pk[1], pk[2], pk[3]);
      }
      const float2 sum = __fadd2_rn(rs[0], rs[1]);
      fence_proxy_async_smem();                  // P, before MMAs and the copy read it
      __syncwarp();
      // the quarter's 32 rows of P (4 KB) to the partner
      if (lane == 0)
        bulk_copy_cluster(p_peer, p_rows, 32 * 128, p_full_peer);
      const float alpha = m_ref != m_old ? exp2_approx(m_old - m_ref) : 1.f;
      st_async(alpha_peer, __float_as_uint(alpha), p_full_peer);
      if (m_ref != m_mine) l_sum *= exp2_approx(m_mine - m_ref);
      m_mine = m_ref;
      l_sum += sum.x + sum.y;
      if (i >= 1 && __any_sync(0xffffffffu, alpha != 1.f)) {   // O to the new reference
        ok = warp_wait(smem_u32(&pv_done[t ^ 1]), ((i - 1) >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
        rescale_o<C::V_HALF>(lane_addr, alpha);
        tc_fence_before();
        __syncwarp();
      }
      if (lane == 0) {
        if (counts) mbar_arrive_expect_tx(smem_u32(&p_full[t]), C::P_TX);
        else mbar_arrive(smem_u32(&p_full[t]));
      }
    }
    // (every arrival that the partner owes has landed before the CTA can leave)
    const int uses = (n - t + 1) / 2;            // tiles of this warp
    if (ok && uses > 0) ok = warp_wait<true>(smem_u32(&p_empty[t]), (uses - 1) & 1);
    if (!ok) {
      abort_s = 1;
      if (lane == 0 && p.status) atomicOr(p.status, kStatusTimeout);
    }
    sSum[t * 128 + hloc] = l_sum;
    sSum[t * 128 + 64 + hloc] = m_mine;
  }
  if (threadIdx.x == 0) mbar_wait(smem_u32(q_bar), 0, nullptr);   // Q has landed
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp < 4 && own) {
    // ---- the heads' sums over both warps' tiles: 1 / sum for both CTAs, LSE
    const int hrow = q * 32 + lane, hloc = hrow & 63;
    const float m0 = sSum[64 + hloc], m1 = sSum[128 + 64 + hloc];
    const float m = fmaxf(m0, m1);
    const float l = (m0 == m ? sSum[hloc] : sSum[hloc] * exp2_approx(m0 - m)) +
                    (m1 == m ? sSum[128 + hloc] : sSum[128 + hloc] * exp2_approx(m1 - m));
    const bool any = n > 0 && !abort_s && !(l <= 0.f);      // (a NaN sum stays visible)
    const float inv = any ? 1.f / l : 0.f;
    const float lse = any ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
    sInv[hrow] = inv;
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(map_to_rank(smem_u32(sInv + hrow), peer)),
                 "f"(inv)
                 : "memory");
    if (hrow < p.h) {
      const int64_t prow = (static_cast<int64_t>(split) * p.row_count + r) * p.h + hrow;
      if (p.part_lse != nullptr) p.part_lse[prow] = lse;
      else p.lse[static_cast<int64_t>(row) * p.h + hrow] = lse;
    }
  }
  __syncwarp();
  cluster_sync();      // both CTAs are done; nothing remote is touched after this
  {
    // ------------------------------------------------------------ epilogue: O / sum
    // The rows are put together in the idle ring (at a pitch of 16 bytes more than a row, so that
    // 8 lanes' 16-byte stores meet all banks) and leave as one bulk copy each.  Stored from the
    // registers, a lane a row, a warp's 16-byte pieces touch 32 rows: 6800 cycles a CTA instead of
    // 2400.
    const int hrow = q * 32 + lane;
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(q * 32) << 16);
    const bool part = p.part_o != nullptr;
    const uint32_t row_bytes = C::V_HALF * (part ? 4 : 2);
    const uint32_t stage = smem_u32(sV) + hrow * (row_bytes + 16);
    const float inv = sInv[hrow];
    for (int c0 = (warp >> 2) * 32; c0 < C::V_HALF; c0 += 128) {
      uint32_t u[32];
      tmem_ld32(lane_addr + c0, u);
      tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < 32; ++j)                // (a row without keys: 0, whatever TMEM holds)
        u[j] = inv != 0.f ? __float_as_uint(__uint_as_float(u[j]) * inv) : 0u;
      if (part) {
#pragma unroll
        for (int j = 0; j < 32; j += 4)
          st_shared_v4(stage + (c0 + j) * 4, u[j], u[j + 1], u[j + 2], u[j + 3]);
      } else {
#pragma unroll
        for (int j = 0; j < 32; j += 8) {
          uint32_t pk[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 two = __floats2bfloat162_rn(__uint_as_float(u[j + 2 * e]),
                                                             __uint_as_float(u[j + 2 * e + 1]));
            pk[e] = *reinterpret_cast<const uint32_t*>(&two);
          }
          st_shared_v4(stage + (c0 + j) * 2, pk[0], pk[1], pk[2], pk[3]);
        }
      }
    }
    fence_proxy_async_smem();                     // the rows, before the copies read them
    named_bar_sync(1 + q, 128);                   // the four warps of this quarter
    if ((lane >> 3) == (warp >> 2)) {             // 8 rows a warp: a copy takes 67 cycles to issue
      if (hrow < p.h) {
        const int64_t orow = static_cast<int64_t>(row) * p.h + hrow;
        const int64_t prow = (static_cast<int64_t>(split) * p.row_count + r) * p.h + hrow;
        void* dst = part ? static_cast<void*>(p.part_o + prow * D_V + c * C::V_HALF)
                         : static_cast<void*>(p.out + orow * D_V + c * C::V_HALF);
        bulk_store_s2g(dst, stage, row_bytes);
      }
      bulk_commit();
      bulk_wait_read_all();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// Merge the splits' partials by their LSE: O = sum_i e^(LSE_i - LSE) O_i, LSE = log sum e^LSE_i.
// One CTA per (row, head); a NaN partial makes the head NaN.  Launched while the attention kernel
// runs, and every load is on its way before the first is used: one token over 2048 keys in 16
// splits takes 16.0 us with the attention, 17.6 with a plain launch.
template <int D_V, int MAX_SPLITS>
__global__ void __launch_bounds__(D_V / 4) dsa_paged_combine_kernel(const PagedMlaParams p) {
  wait_prior_grid();
  const int r = blockIdx.x, hrow = blockIdx.y;
  const int64_t stride = static_cast<int64_t>(p.row_count) * p.h;
  const int64_t base = static_cast<int64_t>(r) * p.h + hrow;
  const int d = threadIdx.x * 4;
  float lse[MAX_SPLITS];
  float4 v[MAX_SPLITS];
#pragma unroll
  for (int s = 0; s < MAX_SPLITS; ++s) {
    const bool in = s < p.splits;
    lse[s] = in ? p.part_lse[s * stride + base] : -INFINITY;
    v[s] = in ? *reinterpret_cast<const float4*>(p.part_o + (s * stride + base) * D_V + d)
              : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  float m = -INFINITY, wsum = 0.f;
#pragma unroll
  for (int s = 0; s < MAX_SPLITS; ++s) m = fmaxf(m, lse[s]);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int s = 0; s < MAX_SPLITS; ++s) {
    if (s >= p.splits) break;
    if (lse[s] == -INFINITY) continue;            // a split without keys
    const float w = expf(lse[s] - m);             // (a NaN LSE stays NaN)
    wsum += w;
    acc.x = fmaf(w, v[s].x, acc.x);
    acc.y = fmaf(w, v[s].y, acc.y);
    acc.z = fmaf(w, v[s].z, acc.z);
    acc.w = fmaf(w, v[s].w, acc.w);
  }
  const bool any = !(wsum <= 0.f);
  const float inv = any ? 1.f / wsum : 0.f;
  const int64_t orow = static_cast<int64_t>(p.row_begin + r) * p.h + hrow;
  const __nv_bfloat162 a = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
  const __nv_bfloat162 c = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
  uint2 pk;
  pk.x = *reinterpret_cast<const uint32_t*>(&a);
  pk.y = *reinterpret_cast<const uint32_t*>(&c);
  *reinterpret_cast<uint2*>(p.out + orow * D_V + d) = pk;
  if (threadIdx.x == 0) p.lse[orow] = any ? m + logf(wsum) : -INFINITY;
}

}  // namespace dsa
