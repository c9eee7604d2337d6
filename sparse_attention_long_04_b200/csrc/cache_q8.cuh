// The paged caches' traffic besides attention: new tokens written (8-bit or bf16 latent rows)
// and ranges of the 8-bit cache read back.  The row format is in q8_row.cuh.
//
// Both kernels move each byte once and compute a handful of instructions per value: HBM is the
// bound for long calls, launch and the dependent loads cu_seqlens -> seq_lens -> block table for
// short ones, which is why the token's own data is loaded before its place in the cache is known.
#pragma once
#include "q8_row.cuh"
#include "rows.cuh"

namespace dsa {

struct CacheWriteParams {
  PagedSeqs s;
  const float* k_new;       // [total_rows, D_I]
  const uint8_t* kv_new;    // [total_rows, D_QK] bf16
  uint8_t* k_cache;         // e4m3 [num_kv_rows, D_I], or blocks with their scales inside
  float* k_scale;           // [num_kv_rows] or null (scales inside the blocks)
  uint8_t* kv_cache;        // [num_kv_rows] rows: 8-bit (Q8Row) or bf16 [D_QK]
  int32_t total_rows;
  int32_t* status;
};

// One warp per new token.  The indexer key: one fp32 scale a token (q8_key, as in the decode
// append).  The latent row: lane l holds values 16 l .. 16 l + 15, so the 8 lanes of
// a 128-value group reduce its largest magnitude in three shuffles and every lane stores one
// 16-byte chunk of codes.
template <int D_I, int D_QK, int D_V, bool kQ8>
__global__ void __launch_bounds__(128) dsa_cache_write_kernel(const CacheWriteParams p) {
  using R = Q8Row<D_QK, D_V>;
  constexpr int PER = D_I / 32;
  constexpr int CHUNKS = D_QK * 2 / 16;        // 16-byte chunks of a bf16 latent row
  constexpr int ROPE_CHUNKS = R::ROPE / 8;
  const int row = blockIdx.x * 4 + static_cast<int>(threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= p.total_rows) return;             // warp-uniform
  // ---- the token's data
  float x[PER];
  const float* ksrc = p.k_new + static_cast<int64_t>(row) * D_I + lane * PER;
  if constexpr (PER == 4) {
    const float4 v = *reinterpret_cast<const float4*>(ksrc);
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) x[i] = ksrc[i];
  }
  const uint4* src = reinterpret_cast<const uint4*>(p.kv_new) + static_cast<int64_t>(row) * CHUNKS;
  uint4 v[3] = {};                             // 8-bit: 16 values and a rotary chunk; else a third
  if constexpr (kQ8) {
    if (lane < D_V / 16) {
      v[0] = src[2 * lane];
      v[1] = src[2 * lane + 1];
    }
    if (lane < ROPE_CHUNKS) v[2] = src[D_V / 8 + lane];
  } else {
#pragma unroll
    for (int i = 0; i < (CHUNKS + 31) / 32; ++i)
      if (lane + 32 * i < CHUNKS) v[i] = src[lane + 32 * i];
  }
  // ---- its cache row
  int b, pos;
  bool bad;
  paged_row(p.s, row, &b, &pos, &bad);
  // a context above max_seqlen would move the token: it is skipped, as one without a place is, and one
  // whose page the caches hold only in part (the indexer would not read it)
  const int64_t dst = bad || pos < 0 ? -1 : paged_phys(p.s, b, pos);
  if (dst < 0 || (p.s.block_table != nullptr && (dst / 64 + 1) * 64 > p.s.num_kv_rows)) {
    if (lane == 0 && p.status) atomicOr(p.status, kStatusBadIndex);
    return;
  }
  // ---- indexer key
  uint32_t packed;
  const float scale = q8_key(x, &packed);
  const int64_t blk = dst / 64, r64 = dst % 64;
  const bool apart = p.k_scale != nullptr;     // scales in their own array
  uint8_t* page = p.k_cache + blk * (64 * (D_I + 4));
  uint8_t* kdst = (apart ? p.k_cache + dst * D_I : page + r64 * D_I) + lane * PER;
  if constexpr (PER == 4) {
    *reinterpret_cast<uint32_t*>(kdst) = packed;
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) kdst[i] = static_cast<uint8_t>(packed >> (8 * i));
  }
  if (lane == 0) *(apart ? p.k_scale + dst : reinterpret_cast<float*>(page + 64 * D_I) + r64) = scale;
  // ---- latent row
  if constexpr (!kQ8) {
    uint4* out = reinterpret_cast<uint4*>(p.kv_cache) + dst * CHUNKS;
#pragma unroll
    for (int i = 0; i < (CHUNKS + 31) / 32; ++i)
      if (lane + 32 * i < CHUNKS) out[lane + 32 * i] = v[i];
  } else {
    uint8_t* out = p.kv_cache + dst * R::BYTES;
    const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
    uint32_t top = 0;                          // largest magnitude, as bf16 bits
#pragma unroll
    for (int i = 0; i < 8; ++i)
      top = max(top, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const bool finite = top < 0x7F80u;
    const int e = finite ? q8_exponent(top) : 0;
    const float inv = exp2_int(-e);
    uint32_t c[4] = {};
    if (finite) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float lo = __uint_as_float(w[i] << 16) * inv;
        const float hi = __uint_as_float(w[i] & 0xFFFF0000u) * inv;
        c[i / 2] |= (q8_code(lo) | (q8_code(hi) << 8)) << (16 * (i & 1));
      }
    }
    if (lane < D_V / 16)
      *reinterpret_cast<uint4*>(out + 16 * lane) = make_uint4(c[0], c[1], c[2], c[3]);
    // the scales' 16 bytes: slot g of group g, unused slots 0
    const float s = finite ? exp2_int(e) : __uint_as_float(0x7FFFFFFFu);
    const float sg = __shfl_sync(0xffffffffu, s, (lane * 8) & 31);
    constexpr int SLOTS = (R::ROPE_OFF - R::SCALE_OFF) / 4;
    if (lane < SLOTS)
      reinterpret_cast<float*>(out + R::SCALE_OFF)[lane] = lane < R::GROUPS ? sg : 0.f;
    if (lane < ROPE_CHUNKS) reinterpret_cast<uint4*>(out + R::ROPE_OFF)[lane] = v[2];
  }
}

struct CacheReadParams {
  PagedSeqs s;
  const uint8_t* kv8;          // 8-bit cache rows
  const int32_t* key_begin;    // [batch] first logical key of each range, or null: 0
  const int32_t* cu_keys;      // [batch + 1] packed output rows of each range
  uint8_t* out;                // [cu_keys[batch], D_QK] bf16
  int32_t total_keys;
  int32_t* status;
};

// One warp per kReadKeys keys: lane l resolves key l, so that the searches and the block-table
// loads of a warp go by once, and every code of the keys is loaded before the first is expanded.
// A lane expands 8 codes into 16 bytes: a warp's stores are whole 512-byte runs.  HBM bounds long
// calls: 223840 keys of (576, 512), 405 MB moved, take 68.1 us, 91% of the measured copy rate; one key a warp,
// with 16-byte code loads and stores at a stride of 32 bytes, took 78.3.
constexpr int kReadKeys = 4;
template <int D_QK, int D_V>
__global__ void __launch_bounds__(256) dsa_cache_read_kernel(const CacheReadParams p) {
  using R = Q8Row<D_QK, D_V>;
  constexpr int CHUNKS = D_V / 8;              // 8-code chunks of a row
  constexpr int PER = (CHUNKS + 31) / 32;      // of them a lane
  constexpr int ROPE_CHUNKS = R::ROPE / 8;     // 16-byte chunks of the rotary dims
  constexpr int ROPE_PER = (kReadKeys * ROPE_CHUNKS + 31) / 32;
  const int r0 = (blockIdx.x * 8 + static_cast<int>(threadIdx.x >> 5)) * kReadKeys;
  const int lane = threadIdx.x & 31;
  const int n = min(p.total_keys, p.cu_keys[p.s.batch]) - r0;   // keys left, may be more than 4
  if (n <= 0) return;                          // warp-uniform
  int64_t my_row = -1;
  if (lane < kReadKeys && lane < n) {
    const int r = r0 + lane;
    const int b = seq_of_row(p.cu_keys, p.s.batch, r);
    const int key = (p.key_begin != nullptr ? p.key_begin[b] : 0) + r - p.cu_keys[b];
    if (key >= 0 && key < min(p.s.seq_lens[b], p.s.max_seqlen)) my_row = paged_phys(p.s, b, key);
    if (my_row < 0 && p.status) atomicOr(p.status, kStatusBadIndex);
  }
  const uint8_t* src[kReadKeys];               // null: a key outside the cache, read as zeros
  uint2 code[kReadKeys][PER];
  float scale[kReadKeys][PER];
  uint4 rope[ROPE_PER];
#pragma unroll
  for (int k = 0; k < kReadKeys; ++k) {
    const int64_t row = __shfl_sync(0xffffffffu, my_row, k);
    src[k] = row >= 0 ? p.kv8 + row * R::BYTES : nullptr;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int ch = lane + 32 * j;
      const bool in = src[k] != nullptr && ch < CHUNKS;
      code[k][j] = in ? __ldcs(reinterpret_cast<const uint2*>(src[k]) + ch) : make_uint2(0, 0);
      scale[k][j] = in ? __ldg(reinterpret_cast<const float*>(src[k] + R::SCALE_OFF) + ch / 16) : 1.f;
    }
  }
#pragma unroll
  for (int j = 0; j < ROPE_PER; ++j) {         // the rotary dims of all keys, one chunk a lane
    const int e = lane + 32 * j;
    const int64_t row = __shfl_sync(0xffffffffu, my_row, min(e / ROPE_CHUNKS, kReadKeys - 1));
    const bool in = row >= 0 && e < kReadKeys * ROPE_CHUNKS;
    rope[j] = in ? __ldcs(reinterpret_cast<const uint4*>(p.kv8 + row * R::BYTES + R::ROPE_OFF) +
                          e % ROPE_CHUNKS)
                 : make_uint4(0, 0, 0, 0);
  }
  uint4* dst = reinterpret_cast<uint4*>(p.out) + static_cast<int64_t>(r0) * (D_QK / 8);
#pragma unroll
  for (int k = 0; k < kReadKeys; ++k) {
    if (k >= n) break;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int ch = lane + 32 * j;
      if (ch < CHUNKS) dst[k * (D_QK / 8) + ch] = q8_expand8(code[k][j], scale[k][j]);
    }
  }
#pragma unroll
  for (int j = 0; j < ROPE_PER; ++j) {
    const int e = lane + 32 * j, k = e / ROPE_CHUNKS;
    if (e < kReadKeys * ROPE_CHUNKS && k < n) dst[k * (D_QK / 8) + CHUNKS + e % ROPE_CHUNKS] = rope[j];
  }
}

}  // namespace dsa
