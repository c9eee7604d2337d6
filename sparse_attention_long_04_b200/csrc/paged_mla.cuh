// MLA attention in MQA mode over the paged caches: single tokens (decode) and chunks of new
// tokens per sequence, over bf16 latent rows or the 8-bit rows of q8_row.cuh.
//
//   l_s = sigma * q[t,h,:] . kv[s,:],  O[t,h,:] = sum_s softmax(l)_s kv[s, 0:D_V],
//   LSE[t,h] = log sum_s exp(l_s),  s over the row's selected keys (idx) or all its keys
//
// Layout of the work: two CTAs per query row (and split of its tiles), CTA v accumulating the
// value dims [v D_V/2, (v+1) D_V/2) in TMEM and computing the full logits of every 64-key tile
// itself, so that the two exchange nothing.  The latent row's 64-dim k-blocks are ordered K part
// (the blocks CTA v needs for the logits only, rotary dims last) then V part (its value blocks);
// Q's blocks follow the same order, the first KBT of them in TMEM, the others in shared memory,
// so that every MMA operand sits at a constant offset from a tile's base.
//
// Issue: one elected lane of a converged warp (elect.sync) issues each tile's MMAs from
// precomputed descriptors.  Issued from an ordinary `lane == 0` branch with the descriptors built
// on the way, an MMA costs 76-90 cycles whatever its size; here 32 (N = 64, A in TMEM), 48
// (A in shared memory, bound by its 6 KB of operand reads) and 128 (N = 256), measured with all
// SMs issuing.  A 64-key tile is then 20 x 32 + 16 x 48 + 4 x 128 = 1920 cycles of tensor pipe
// at (576, 512).
//
// 8-bit rows: the gather warps read the codes into registers, expand them to bf16 (exactly: the
// scales are powers of two) and store them into the same swizzled tiles the bf16 gather fills
// with cp.async; the rotary dims are bf16 in both caches and always come by cp.async.
//
// Warp roles (512 threads): warp 0 issues the MMAs, warp 1 owns TMEM, warps 4-7 Q into TMEM, softmax and
// epilogue (thread = head), warps 8-11 the K part and warps 12-15 the V part of every tile.
// Without idx the keys are every prior key; a 64-key tile is then one page, and the pages of a
// split's tiles are resolved up front (kMaxDenseTiles of them).
#pragma once
#include "q8_row.cuh"
#include "rows.cuh"
#include "sparse_mla.cuh"

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

// Rings of one CTA: the K part's value blocks in one slot (freed as soon as their MMAs have run,
// refilled while the V part's run), the rotary block in two, the V part in three (a slot is held
// until PV, and the next use needs it only when the third QK after comes to its V part).
template <int D_QK, int D_V>
struct PagedCfg {
  static constexpr int KB_ALL = (D_QK + 63) / 64;     // 64-dim k-blocks of a latent row
  static constexpr int V_HALF = D_V / 2;              // value dims per CTA
  static constexpr int VKB = V_HALF / 64;             // value blocks per CTA (V part)
  static constexpr int NK = KB_ALL - VKB - 1;         // value blocks of the other CTA (K part)
  static constexpr int BN = 64;                       // keys per tile
  static constexpr int R_SLOTS = 2, V_SLOTS = 3;
  static constexpr int MAX_TILES = 32;                // topk <= 2048
  static constexpr int THREADS = 512;
  // TMEM: O, S, P (bf16), then the rotary and K-part blocks of Q and as many more as fit
  static constexpr int S_COL = V_HALF;
  static constexpr int P_COL = S_COL + BN;
  static constexpr int Q_COL = P_COL + BN / 2;
  static constexpr int KBT_MAX = (512 - Q_COL) / 32;
  static constexpr int KBT = KB_ALL < KBT_MAX ? KB_ALL : KBT_MAX;   // Q blocks in TMEM
  static constexpr int KBS = KB_ALL - KBT;                            // Q blocks in smem
  static constexpr int TMEM_COLS = Q_COL + KBT * 32 <= 256 ? 256 : 512;
  static constexpr int KB_BYTES = BN * 128;                           // one k-block of a tile
  static constexpr int RING_BYTES = (NK + R_SLOTS + V_SLOTS * VKB) * KB_BYTES;
  static constexpr int Q_KB_BYTES = 128 * 128;                        // one k-block of Q
  static constexpr int Q_SMEM_BYTES = KBS * Q_KB_BYTES;
  static constexpr int SMEM_USED = 1024 + Q_SMEM_BYTES + RING_BYTES + MAX_TILES * BN * 4 +
                                   MAX_TILES * 12 + 256;
  // at least 116 KB, so that one CTA runs per SM (its TMEM allocation never waits)
  static constexpr int SMEM_BYTES = SMEM_USED > 116 * 1024 ? SMEM_USED : 116 * 1024;
  static_assert(V_HALF % 64 == 0 && V_HALF <= 256, "PV MMA N");
  static_assert(NK == VKB, "both parts hold as many value blocks");
  static_assert(KBT >= NK + 1, "the K part's Q blocks live in TMEM");
  static_assert(Q_COL + KBT * 32 <= 512, "TMEM columns");
  static_assert(KBT * Q_KB_BYTES <= RING_BYTES, "Q staging fits the gather rings");
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
};

constexpr int kMaxDenseTiles = 2048;   // tiles of one split without idx

// True in one lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// Whole-warp wait for phase `parity` of `bar`: every lane polls (one broadcast access) without a
// suspend-time hint, which a completed phase answers in 14 cycles against 46 with the hint and 195
// for warp_mbar_wait's poll by lane 0 and shuffle.  The clock and the abort flag are looked at
// once in 64 polls; all lanes return the same result.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity,
                                          const volatile int* abort) {
  uint32_t ok = 0;
  uint64_t t0 = 0;
#pragma unroll 1
  for (uint32_t it = 1;; ++it) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (ok) break;
    if ((it & 63u) == 0) {
      if (abort != nullptr && *abort) break;
      const uint64_t now = global_timer_ns();
      if (t0 == 0) t0 = now;
      else if (now - t0 > kWaitLimitNs) break;
    }
  }
  return __all_sync(0xffffffffu, ok) != 0;
}

// 2^x, results below the normal range flushed to 0 (a probability that small adds nothing).
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Grid: x = 2 * row + v, y = split.  Tile sizes, rings and TMEM columns are MlaCfg's.
template <int D_QK, int D_V, bool kQ8>
__global__ void __launch_bounds__(512, 1)
    dsa_paged_mla_kernel(const __grid_constant__ CUtensorMap q_map, const PagedMlaParams p) {
  using C = PagedCfg<D_QK, D_V>;
  using R = Q8Row<D_QK, D_V>;
  constexpr int ROW_BYTES = kQ8 ? R::BYTES : D_QK * 2;
  static_assert(R::ROPE <= 64 && D_V % 64 == 0, "rotary dims fill (part of) the last k-block");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* sQ = smem;                                           // [KBS][128 heads][128 B]
  uint8_t* sRing = sQ + C::Q_SMEM_BYTES;                        // gather rings (Q staging first)
  uint8_t* sK = sRing;                                          // [NK k-blocks]
  uint8_t* sR = sK + C::NK * C::KB_BYTES;                       // [R_SLOTS] rotary k-blocks
  uint8_t* sV = sR + C::R_SLOTS * C::KB_BYTES;                  // [V_SLOTS][VKB k-blocks]
  // selected: the physical row of every key; dense: the first physical row of every tile
  int32_t* sPhys = reinterpret_cast<int32_t*>(sRing + C::RING_BYTES);             // [2048]
  uint64_t* sMask = reinterpret_cast<uint64_t*>(sPhys + C::MAX_TILES * C::BN);   // [32]
  int32_t* sTiles = reinterpret_cast<int32_t*>(sMask + C::MAX_TILES);            // [32]
  uint64_t* bars = reinterpret_cast<uint64_t*>(sTiles + C::MAX_TILES);
  uint64_t* k_full = bars;           // every K-part thread
  uint64_t* k_empty = bars + 1;      // commit of the K part's MMAs
  uint64_t* r_full = bars + 2;       // [2] every K-part thread (rotary copies landed)
  uint64_t* r_empty = bars + 4;      // [2] the same commit
  uint64_t* v_full = bars + 6;       // [3] every V-part thread
  uint64_t* v_empty = bars + 9;      // [3] PV commit
  uint64_t* s_full = bars + 12;       // QK commit
  uint64_t* s_empty = bars + 13;      // 4 softmax warps
  uint64_t* p_full = bars + 14;      // 4 softmax warps
  uint64_t* pv_done = bars + 15;     // PV commit
  uint64_t* mma_fin = bars + 16;     // every MMA of this CTA completed
  uint64_t* q_bar = bars + 17;       // 1 arrival + Q bytes
  __shared__ uint32_t tmem_base_s;
  __shared__ int abort_s;
  __shared__ int n_act_s;
  static_assert(kMaxDenseTiles <= C::MAX_TILES * C::BN, "dense tiles fit the key array");

  wait_prior_grid();   // (launched early: the indices come from the previous kernel)
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int vh = static_cast<int>(blockIdx.x & 1u);   // value half
  const int split = blockIdx.y;
  const int r = blockIdx.x >> 1;
  const int row = p.row_begin + r;
  const bool dense = p.idx == nullptr;
  const int n_tiles_all = p.topk / C::BN;

  // ---- row geometry; the selected keys' indices (8 per thread of warps 8-15) are loaded first,
  // so that their latency overlaps it and the set-up
  constexpr int KPT = C::MAX_TILES * C::BN / 256;
  int v[KPT];
  if (warp >= 8 && !dense) {
    const int32_t* irow = p.idx + static_cast<int64_t>(r) * p.topk;
#pragma unroll
    for (int j = 0; j < KPT; ++j) {
      const int e = static_cast<int>(threadIdx.x) - 256 + 256 * j;
      v[j] = e < p.topk ? irow[e] : -1;
    }
  }
  int b, pos;
  bool bad_row;
  paged_row(p.s, row, &b, &pos, &bad_row);
  const int n_keys = max(pos + 1, 0);
  if (bad_row && threadIdx.x == 0 && p.status) atomicOr(p.status, kStatusBadIndex);

  if (threadIdx.x == 0) {
    mbar_init(smem_u32(k_full), 128);
    mbar_init(smem_u32(k_empty), 1);
    for (int i = 0; i < C::R_SLOTS; ++i) {
      mbar_init(smem_u32(&r_full[i]), 128);
      mbar_init(smem_u32(&r_empty[i]), 1);
    }
    for (int i = 0; i < C::V_SLOTS; ++i) {
      mbar_init(smem_u32(&v_full[i]), 128);
      mbar_init(smem_u32(&v_empty[i]), 1);
    }
    mbar_init(smem_u32(s_full), 1);
    mbar_init(smem_u32(s_empty), 4);
    mbar_init(smem_u32(p_full), 4);
    mbar_init(smem_u32(pv_done), 1);
    mbar_init(smem_u32(mma_fin), 1);
    mbar_init(smem_u32(q_bar), 1);
    abort_s = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(smem_u32(&tmem_base_s), C::TMEM_COLS);
  __syncthreads();
  if (threadIdx.x == 0) {
    // ---- Q, in the order rotary, K part, V part: KBT blocks into the (still idle) rings, the rest
    // into sQ; h rows a block (lanes past h hold whatever the staging area held and are never written)
    const uint32_t kb_bytes = static_cast<uint32_t>(p.h) * 128u;
    tma_prefetch_desc(&q_map);
    mbar_arrive_expect_tx(smem_u32(q_bar), C::KB_ALL * kb_bytes);
    for (int j = 0; j < C::KB_ALL; ++j) {
      const int v0 = vh * C::VKB;
      const int kb = j == 0 ? C::KB_ALL - 1
                   : j > C::NK ? v0 + j - 1 - C::NK
                               : (j - 1 < v0 ? j - 1 : j - 1 + C::VKB);
      uint8_t* dst = j < C::KBT ? sRing + j * C::Q_KB_BYTES : sQ + (j - C::KBT) * C::Q_KB_BYTES;
      tma_load_2d(smem_u32(dst), &q_map, smem_u32(q_bar), kb * 128, r * p.h);
    }
  }
  bool bad_idx = false;
  if (warp >= 8 && !dense) {
    // ---- every selected key -> physical row (or -1), all block-table loads in flight together
    int64_t phys[KPT];
#pragma unroll
    for (int j = 0; j < KPT; ++j) {
      phys[j] = -1;
      if (v[j] >= 0 && v[j] < n_keys)
        phys[j] = paged_phys(p.s, b, v[j]);
      bad_idx |= v[j] >= 0 && phys[j] < 0;
    }
#pragma unroll
    for (int j = 0; j < KPT; ++j) {
      const int e = static_cast<int>(threadIdx.x) - 256 + 256 * j;
      if (e < p.topk) sPhys[e] = static_cast<int32_t>(phys[j]);
    }
  }
  __syncthreads();
  if (warp >= 8 && !dense) {
    // ---- per tile: the valid-key mask; invalid keys borrow the tile's first valid row
    for (int tt = warp - 8; tt < n_tiles_all; tt += 8) {
      int32_t* ph = sPhys + tt * C::BN;
      const int32_t a0 = ph[lane], a1 = ph[32 + lane];
      const uint32_t lo = __ballot_sync(0xffffffffu, a0 >= 0);
      const uint32_t hi = __ballot_sync(0xffffffffu, a1 >= 0);
      const uint64_t m = (static_cast<uint64_t>(hi) << 32) | lo;
      if (m != 0) {
        const int32_t fb = ph[__ffsll(static_cast<long long>(m)) - 1];
        __syncwarp();
        if (a0 < 0) ph[lane] = fb;
        if (a1 < 0) ph[32 + lane] = fb;
      }
      if (lane == 0) sMask[tt] = m;
    }
  }
  if (warp == 8 && dense) {
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
  __syncthreads();
  if (warp == 0 && lane == 0 && !dense) {
    // ---- the active tiles of this split, identical in both CTAs of the row
    int cnt = 0;
    for (int t = 0; t < n_tiles_all; ++t)
      if (sMask[t] != 0) sTiles[cnt++] = t;
    const int per = (cnt + p.splits - 1) / p.splits;
    const int t0 = min(cnt, split * per);
    const int t1 = min(cnt, t0 + per);
    for (int i = t0; i < t1; ++i) sTiles[i - t0] = sTiles[i];
    n_act_s = t1 - t0;
  }
  if (warp >= 4 && warp < 8) {
    // ---- Q blocks [0, KBT) from the staging area into TMEM: head = lane, dim d in column
    // Q_COL + d / 2
    const int hrow = (warp & 3) * 32 + lane;
    const uint32_t lane_addr = tmem_base_s + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    if (!(warp_wait(smem_u32(q_bar), 0, &abort_s))) {
      abort_s = 1;
      if (p.status) atomicOr(p.status, kStatusTimeout);
    } else {
      for (int kb = 0; kb < C::KBT; ++kb) {
        uint32_t u[32];
        const uint8_t* src = sRing + kb * C::Q_KB_BYTES;
#pragma unroll
        for (int ch = 0; ch < 8; ++ch) {
          const uint4 q4 = *reinterpret_cast<const uint4*>(src + sw128_offset(hrow, ch));
          u[4 * ch + 0] = q4.x;
          u[4 * ch + 1] = q4.y;
          u[4 * ch + 2] = q4.z;
          u[4 * ch + 3] = q4.w;
        }
        tmem_st32(lane_addr + C::Q_COL + kb * 32, u);
      }
      tmem_wait_st();
    }
  }
  tc_fence_before();
  __syncthreads();   // the staging area is free for the gather rings from here on
  tc_fence_after();
  const uint32_t tmem = tmem_base_s;
  const int n = abort_s ? 0 : n_act_s;
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

  if (warp == 0) {
    // ------------------------------------------------------------ MMA issuer
    // QK(i) is issued before PV(i - 1), so that the tensor pipe runs PV(i - 1) while the softmax
    // warps read S(i) out of its single buffer (and QK(i + 1) still has to wait for them).
    constexpr uint32_t idesc_qk = idesc_f32acc(1 /* bf16 */, 128, C::BN, 0, 0);
    constexpr uint32_t idesc_pv = idesc_f32acc(1, 128, C::V_HALF, 0, 1);
    const uint64_t qd = sdesc_sw128(smem_u32(sQ), 16, 1024);
    bool ok = n == 0 || warp_wait(smem_u32(q_bar), 0, &abort_s);
    const uint64_t kd = sdesc_sw128(smem_u32(sK), 16, 1024);
    int vs = 0, vs1 = 0;            // V slots of tiles i and i - 1
    uint32_t vph = 0;
    for (int i = 0; i <= n && ok; ++i) {
      if (i < n) {
        const int rs = i & 1;
        const uint64_t rd = sdesc_sw128(smem_u32(sR + rs * C::KB_BYTES), 16, 1024);
        const uint64_t vd = sdesc_sw128(smem_u32(sV + vs * (C::VKB * C::KB_BYTES)), 16, 1024);
        ok = warp_wait(smem_u32(&r_full[rs]), (i >> 1) & 1, &abort_s) &&
             warp_wait(smem_u32(k_full), i & 1, &abort_s) &&
             (i == 0 || warp_wait(smem_u32(s_empty), (i - 1) & 1, &abort_s));
        if (!ok) break;
        tc_fence_after();
        fence_proxy_async_smem();   // the rows were written by cp.async and ordinary stores
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            umma_bf16_ts(tmem + C::S_COL, tmem + C::Q_COL + k * 8, rd + k * 2, idesc_qk, k != 0);
#pragma unroll
          for (int k = 0; k < 4 * C::NK; ++k)
            umma_bf16_ts(tmem + C::S_COL, tmem + C::Q_COL + 32 + k * 8,
                         kd + ((k / 4) * C::KB_BYTES + (k % 4) * 32) / 16, idesc_qk, 1u);
          umma_commit(smem_u32(k_empty));
          umma_commit(smem_u32(&r_empty[rs]));
        }
        __syncwarp();
        ok = warp_wait(smem_u32(&v_full[vs]), vph, &abort_s);
        if (!ok) break;
        tc_fence_after();
        fence_proxy_async_smem();
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < 4 * C::VKB; ++k) {
            const int j = 1 + C::NK + k / 4;         // Q block
            const uint64_t bd = vd + ((k / 4) * C::KB_BYTES + (k % 4) * 32) / 16;
            if (j < C::KBT)
              umma_bf16_ts(tmem + C::S_COL, tmem + C::Q_COL + j * 32 + (k % 4) * 8, bd, idesc_qk,
                           1u);
            else
              umma_bf16(tmem + C::S_COL,
                        qd + ((j - C::KBT) * C::Q_KB_BYTES + (k % 4) * 32) / 16, bd, idesc_qk, 1u);
          }
          umma_commit(smem_u32(s_full));
        }
        __syncwarp();
      }
      if (i > 0) {
        const uint64_t vd = sdesc_sw128(smem_u32(sV + vs1 * (C::VKB * C::KB_BYTES)), C::KB_BYTES,
                                        1024);
        ok = warp_wait(smem_u32(p_full), (i - 1) & 1, &abort_s);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < C::BN / 16; ++k)
            umma_bf16_ts(tmem, tmem + C::P_COL + k * 8, vd + k * 16 * 128 / 16, idesc_pv,
                         i > 1 || k != 0);
          umma_commit(smem_u32(&v_empty[vs1]));
          umma_commit(smem_u32(pv_done));
        }
        __syncwarp();
      }
      vs1 = vs;
      if (++vs == C::V_SLOTS) {
        vs = 0;
        vph ^= 1u;
      }
    }
    if (!ok) {
      abort_s = 1;
      if (lane == 0 && p.status) atomicOr(p.status, kStatusTimeout);
    }
    __syncwarp();
    if (elect_one()) umma_commit(smem_u32(mma_fin));   // no MMA may outlive the CTA
    __syncwarp();
    warp_wait(smem_u32(mma_fin), 0, nullptr);
  } else if (warp >= 8) {
    // ------------------------------------------------------------ gather producers
    // Warp 8 + 4 part + w fills rows [16w, 16w + 16) of each tile: part 0 the K part (and the
    // rotary block), part 1 the V part.
    const int part = (warp - 8) >> 2;
    const int pw = (warp - 8) & 3;
    const int ch = lane & 7;                    // 16-byte chunk of a 128-byte row block
    const int rsub = lane >> 3;                 // rows rsub, rsub + 4, rsub + 8, rsub + 12
    const int kb0 = (part == 0) == (vh == 0) ? C::VKB : 0;   // the part's first latent block
    // a block of bf16 rows straight from the cache, its chunks past `valid` zeros
    auto copy_block = [&](uint8_t* dst, int i, int byte, int valid) {
      const bool in = ch < valid;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int rr = pw * 16 + rsub + 4 * j;
        const uint8_t* src = p.kv + phys_of(i, rr) * ROW_BYTES + byte + ch * 16;
        cp_async_16(smem_u32(dst) + sw128_offset(rr, ch), in ? src : p.kv, in ? 16u : 0u);
      }
    };
    // 8-bit codes: lane = 16-code chunk lane % 4 of rows lane / 4 and lane / 4 + 8, every value block
    // of the part.  Eight lanes, two neighbouring rows, then store to the eight different 16-byte
    // columns of a swizzled tile (eight lanes on one row would meet two to a column: 8.1 instead
    // of 4 wavefronts a store).  Two register sets take turns: the set just stored is loaded with
    // the codes and scales of two tiles on, so that their latency (HBM's, where the cache is
    // large) goes by under a whole tile.
    constexpr int GP = (C::VKB + 1) / 2;         // scales of a row's part (128 values, 2 blocks)
    struct CodeSet {
      uint4 code[2][C::VKB];
      float scale[2][GP];
    };
    const int cl = lane & 3, rl = pw * 16 + (lane >> 2);
    auto load_set = [&](CodeSet& x, int i) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const uint8_t* src = p.kv + phys_of(i, rl + 8 * q) * ROW_BYTES;
#pragma unroll
        for (int g = 0; g < GP; ++g)
          x.scale[q][g] = __ldg(reinterpret_cast<const float*>(src + R::SCALE_OFF) + kb0 / 2 + g);
#pragma unroll
        for (int ks = 0; ks < C::VKB; ++ks)
          x.code[q][ks] = __ldg(reinterpret_cast<const uint4*>(src + (kb0 + ks) * 64) + cl);
      }
    };
    auto store_set = [&](const CodeSet& x, uint8_t* dst) {
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int ks = 0; ks < C::VKB; ++ks) {
          uint8_t* at = dst + ks * C::KB_BYTES;
          uint4 lo, hi;
          q8_expand16(x.code[q][ks], x.scale[q][ks / 2], lo, hi);
          *reinterpret_cast<uint4*>(at + sw128_offset(rl + 8 * q, 2 * cl)) = lo;
          *reinterpret_cast<uint4*>(at + sw128_offset(rl + 8 * q, 2 * cl + 1)) = hi;
        }
    };
    bool ok = true;
    int vs = 0;
    uint32_t vph = 1;                            // (the first use of each slot does not wait)
    // tile i: its slot waited for, filled, and the barrier told
    auto fill = [&](CodeSet& x, int i) -> bool {
      uint8_t* dst;
      uint64_t* full;
      if (part == 0) {
        const int rs = i & 1;
        if (i >= C::R_SLOTS &&
            !warp_wait(smem_u32(&r_empty[rs]), ((i >> 1) - 1) & 1, &abort_s))
          return false;
        copy_block(sR + rs * C::KB_BYTES, i, kQ8 ? R::ROPE_OFF : 2 * D_V, R::ROPE / 8);
        cp_async_arrive_noinc(smem_u32(&r_full[rs]));
        if (i >= 1 && !warp_wait(smem_u32(k_empty), (i - 1) & 1, &abort_s)) return false;
        dst = sK;
        full = k_full;
      } else {
        if (i >= C::V_SLOTS && !warp_wait(smem_u32(&v_empty[vs]), vph, &abort_s)) return false;
        dst = sV + vs * (C::VKB * C::KB_BYTES);
        full = &v_full[vs];
        if (++vs == C::V_SLOTS) {
          vs = 0;
          vph ^= 1u;
        }
      }
      if constexpr (kQ8) {
        store_set(x, dst);
        fence_proxy_async_smem();              // this thread's stores, before the MMAs read them
        mbar_arrive(smem_u32(full));
        if (i + 2 < n) load_set(x, i + 2);
      } else {
#pragma unroll
        for (int ks = 0; ks < C::VKB; ++ks)
          copy_block(dst + ks * C::KB_BYTES, i, (kb0 + ks) * 128, 8);
        cp_async_arrive_noinc(smem_u32(full));
      }
      return true;
    };
    CodeSet set0, set1;
    if constexpr (kQ8) {
      if (n > 0) load_set(set0, 0);
      if (n > 1) load_set(set1, 1);
    }
    for (int i = 0; i < n && ok; i += 2) {
      ok = fill(set0, i);
      if (ok && i + 1 < n) ok = fill(set1, i + 1);
    }
    if (!ok) {
      abort_s = 1;
      if (p.status) atomicOr(p.status, kStatusTimeout);
    }
    cp_async_wait_all();   // nothing may still be writing this CTA's shared memory at exit
  } else if (warp >= 4) {
    // ------------------------------------------------------------ softmax + epilogue
    const int hrow = (warp & 3) * 32 + lane;    // head = TMEM lane
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    float m_ref = -INFINITY, l_sum = 0.f;
    bool ok = !abort_s;
    for (int i = 0; i < n && ok; ++i) {
      ok = (warp_wait(smem_u32(s_full), i & 1, &abort_s));
      if (!ok) break;
      tc_fence_after();
      uint32_t su[2][32];                       // S of keys [32 hh, 32 hh + 32)
      tmem_ld32(lane_addr + C::S_COL, su[0]);
      tmem_ld32(lane_addr + C::S_COL + 32, su[1]);
      tmem_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(s_empty));
      const uint64_t vmask = mask_of(i);
      if (vmask != ~0ull) {
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const uint32_t vb = static_cast<uint32_t>(vmask >> (32 * hh));
#pragma unroll
          for (int j = 0; j < 32; ++j)           // invalid keys: -inf, so p = 0 below
            if (!((vb >> j) & 1u)) su[hh][j] = 0xFF800000u;
        }
      }
      // the tile max of the unscaled logits (sigma log2 e > 0), as 8 independent partial maxima
      float mm[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) mm[q] = __uint_as_float(su[0][q]);
#pragma unroll
      for (int j = 8; j < 64; j += 16)
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float x = __uint_as_float(su[(j + q) / 32][(j + q) % 32]);
          const int j2 = j + 8 + q;
          mm[q] = j2 < 64 ? fmaxf(fmaxf(mm[q], x), __uint_as_float(su[j2 / 32][j2 % 32]))
                          : fmaxf(mm[q], x);
        }
      const float m_tile =
          fmaxf(fmaxf(fmaxf(mm[0], mm[1]), fmaxf(mm[2], mm[3])),
                fmaxf(fmaxf(mm[4], mm[5]), fmaxf(mm[6], mm[7]))) * p.scale_log2;
      // the reference moves only when a tile beats it by 2^8: p and the sums stay far inside
      // fp32 (and bf16) either way
      const bool need = m_tile > m_ref + 8.0f;
      float alpha = 1.f;
      if (need) {
        alpha = exp2_approx(m_ref - m_tile);
        l_sum *= alpha;
        m_ref = m_tile;
      }
      // p = 2^(sigma log2e s - m_ref); the denominator sums the fp32 probabilities, only the PV
      // operand is rounded (bf16: the MMA's operand type)
      // (two keys to an instruction: the scaling FMA and the sums are packed fp32 pairs)
      float2 rs[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) rs[q] = make_float2(0.f, 0.f);
      const float2 sc2 = make_float2(p.scale_log2, p.scale_log2), nm2 = make_float2(-m_ref, -m_ref);
      uint32_t pk[2][16];
#pragma unroll
      for (int hh = 0; hh < 2; ++hh)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float2 x = __ffma2_rn(make_float2(__uint_as_float(su[hh][2 * e]),
                                                  __uint_as_float(su[hh][2 * e + 1])), sc2, nm2);
          const float2 pr = make_float2(exp2_approx(x.x), exp2_approx(x.y));
          rs[e & 3] = __fadd2_rn(rs[e & 3], pr);
          const __nv_bfloat162 two = __float22bfloat162_rn(pr);
          pk[hh][e] = *reinterpret_cast<const uint32_t*>(&two);
        }
      const float2 r01 = __fadd2_rn(__fadd2_rn(rs[0], rs[1]), __fadd2_rn(rs[2], rs[3]));
      l_sum += r01.x + r01.y;
      // P and O are free once PV(i-1) has completed
      if (i >= 1) {
        ok = (warp_wait(smem_u32(pv_done), (i - 1) & 1, &abort_s));
        if (!ok) break;
        tc_fence_after();
        if (__any_sync(0xffffffffu, need)) {       // O to the new reference
          for (int c0 = 0; c0 < C::V_HALF; c0 += 32) {
            uint32_t u[32];
            tmem_ld32(lane_addr + c0, u);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) u[j] = __float_as_uint(__uint_as_float(u[j]) * alpha);
            tmem_st32(lane_addr + c0, u);
          }
        }
      }
      tmem_st16(lane_addr + C::P_COL, pk[0]);
      tmem_st16(lane_addr + C::P_COL + 16, pk[1]);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(p_full));
    }
    if (!ok) {
      abort_s = 1;
      if (p.status) atomicOr(p.status, kStatusTimeout);
    }
    // ---- epilogue
    const bool write = hrow < p.h;
    const int64_t orow = static_cast<int64_t>(row) * p.h + hrow;
    if (ok && n > 0)
      ok = (warp_wait(smem_u32(pv_done), (n - 1) & 1, &abort_s));
    tc_fence_after();
    const bool any = ok && n > 0 && !(l_sum <= 0.f);   // (a NaN sum stays visible)
    const float inv_l = any ? 1.f / l_sum : 0.f;
    const float lse_v = any ? (m_ref + log2f(l_sum)) * 0.69314718055994531f : -INFINITY;
    const int64_t prow = (static_cast<int64_t>(split) * p.row_count + r) * p.h + hrow;
    float* po = p.part_o != nullptr ? p.part_o + prow * D_V + vh * C::V_HALF : nullptr;
    for (int c0 = 0; c0 < C::V_HALF; c0 += 32) {
      float o[32];
      if (ok && n > 0) {                          // (warp-uniform: the TMEM load is collective)
        uint32_t u[32];
        tmem_ld32(lane_addr + c0, u);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 32; ++j) o[j] = any ? __uint_as_float(u[j]) * inv_l : 0.f;
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) o[j] = 0.f;
      }
      if (!write) continue;
      if (po != nullptr) {
#pragma unroll
        for (int j = 0; j < 32; j += 4)
          *reinterpret_cast<float4*>(po + c0 + j) = make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
      } else {
        __nv_bfloat16* dst = p.out + orow * D_V + vh * C::V_HALF + c0;
#pragma unroll
        for (int j = 0; j < 32; j += 8) {
          uint32_t pk[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 two = __floats2bfloat162_rn(o[j + 2 * e], o[j + 2 * e + 1]);
            pk[e] = *reinterpret_cast<const uint32_t*>(&two);
          }
          *reinterpret_cast<uint4*>(dst + j) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
        }
      }
    }
    if (write && vh == 0) {
      if (p.part_lse != nullptr) p.part_lse[prow] = lse_v;
      else p.lse[orow] = lse_v;
    }
  }
  if (threadIdx.x == 0) mbar_wait(smem_u32(q_bar), 0, nullptr);   // Q has landed
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// Merge the splits' partials by their LSE: O = sum_i e^(LSE_i - LSE) O_i, LSE = log sum e^LSE_i.
// One CTA per (row, head); a NaN partial makes the head NaN.
template <int D_V>
__global__ void __launch_bounds__(D_V / 4) dsa_paged_combine_kernel(const PagedMlaParams p) {
  const int r = blockIdx.x, hrow = blockIdx.y;
  const int64_t stride = static_cast<int64_t>(p.row_count) * p.h;
  const int64_t base = static_cast<int64_t>(r) * p.h + hrow;
  float m = -INFINITY, wsum = 0.f;
  for (int s = 0; s < p.splits; ++s) m = fmaxf(m, p.part_lse[s * stride + base]);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  const int d = threadIdx.x * 4;
  for (int s = 0; s < p.splits; ++s) {
    const float lse = p.part_lse[s * stride + base];
    const float w = lse == -INFINITY ? 0.f : expf(lse - m);   // a NaN LSE stays NaN
    const float4 v = *reinterpret_cast<const float4*>(p.part_o + (s * stride + base) * D_V + d);
    wsum += w;
    acc.x = fmaf(w, v.x, acc.x);
    acc.y = fmaf(w, v.y, acc.y);
    acc.z = fmaf(w, v.z, acc.z);
    acc.w = fmaf(w, v.w, acc.w);
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
