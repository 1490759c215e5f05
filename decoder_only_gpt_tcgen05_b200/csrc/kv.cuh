// The quantised key/value cache: tile geometry, the ragged batch, and the small device helpers that
// its kernels (kv_cache.cu, kv_select.cu, kv_attention.cu) share.
//
// A cache block holds 64 tokens.  For each kv head it is one contiguous tile of two records of 32
// tokens, so a warp fetches a record (keys, values and scales) with one bulk copy:
//
//   [32 key rows][32 value rows][32 x NG key scales][32 x NG value scales]
//
// Codes are unsigned with the zero at Z (8 or 128), value = scale * (code - Z); a scale covers 64
// dims (4 bits) or the whole row (8 bits).  Within a record the code bytes lie in the order in which
// the attention kernel's mma fragments take them, so every shared-memory read is 8 or 16 contiguous
// bytes a lane without bank conflicts and needs no shuffle:
//
//   keys    lane (key i mod 8, c = lane mod 4) holds the row's 32-bit words c, c + 4, c + 8, ...
//   values  lane (r, c) holds, for the keys 2c, 2c + 1, 2c + 8, 2c + 9 of 16, the octets (8 dims)
//           r, r + 8 of the row: the k pairs and the rows of an m16n8k16 A fragment of V^T
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "gpt_ops.h"
#include "host.cuh"
#include "kernels.cuh"
#include "ptx.cuh"

namespace gptk {

constexpr int kKvBlock = GPT_KV_BLOCK;  // tokens of a block
constexpr int kKvRec = 32;              // tokens of a record

template <int BITS_, int HD_>
struct KvGeom {
  static constexpr int BITS = BITS_, HD = HD_;
  static constexpr int ROWB = HD * BITS / 8;             // code bytes of a row
  static constexpr int NG = BITS == 4 ? HD / 64 : 1;     // scales of a row
  static constexpr int KB = ROWB / 4;                    // key bytes of a lane and row
  static constexpr int KP = KB < 16 ? KB : 16;           // ... contiguous ones
  static constexpr int VB = ROWB / 8;                    // value bytes of a lane and key
  static constexpr int KCODES = 0;
  static constexpr int VCODES = kKvRec * ROWB;
  static constexpr int KSCALE = 2 * kKvRec * ROWB;
  static constexpr int VSCALE = KSCALE + kKvRec * NG * 2;
  static constexpr int REC = VSCALE + kKvRec * NG * 2;   // bytes of a record, a multiple of 64
  static constexpr int TILE = 2 * REC;
  static constexpr int Z = 1 << (BITS - 1);
  static constexpr int TOP = Z - 1;                      // largest |code - Z| written

  // byte offset in the record of word w (of the row's natural order) of key i
  static __host__ __device__ constexpr int key_word(int i, int w) {
    const int c = w & 3, y = (w >> 2) * 4;
    return (i >> 4) * 16 * ROWB + (y / KP) * 64 * KP + (i & 15) * 4 * KP + c * KP + y % KP;
  }
  // byte offset in the record of octet o (BITS bytes) of value i
  static __host__ __device__ constexpr int value_octet(int i, int o) {
    const int ii = i & 15, lane = 4 * (o & 7) + ((ii & 7) >> 1);
    const int z = ((ii & 1) + 2 * (ii >> 3)) * VB + (o >> 3) * BITS;
    return VCODES + (i >> 4) * 16 * ROWB + (z >> 4) * 512 + lane * 16 + (z & 15);
  }
};

// These kernels are launched so that they may start while the kernel before them finishes (launch_pdl):
// what they read may still be being written then, so after pdl_wait() it is read by ordinary loads, never
// by non-coherent ones.

// The ragged batch of a call (gpt_kv_batch), with the number of rows of the row tensors.
struct KvRows {
  const int* table;
  const int* lens;
  const int* cu;  // may be null: one row per sequence
  int B, W, max_new, M;
};

// Sequence b of the batch: n rows from row0 on, the last of which is the token at position len - 1.
// ok = false for a sequence whose numbers are out of range (nothing of it may be touched).
struct KvSeq {
  int row0, n, len;
  bool ok;
};
__device__ __forceinline__ KvSeq kv_seq(const KvRows& r, int b) {
  KvSeq s;
  s.row0 = r.cu ? r.cu[b] : b;
  const long long n = r.cu ? (long long)r.cu[b + 1] - s.row0 : 1;
  s.len = r.lens[b];
  s.ok = n >= 0 && n <= r.max_new && s.row0 >= 0 && s.row0 + n <= r.M && s.len >= n &&
         s.len <= (long long)r.W * kKvBlock;
  s.n = s.ok ? (int)n : 0;
  return s;
}

// Reports sequences out of range where the work is dealt by rows, which such a sequence may not have.
__device__ __forceinline__ void kv_report_bad(const KvRows& r, const DevCtl& ctl, unsigned int site) {
  for (int b = threadIdx.x; b < r.B; b += blockDim.x)
    if (!kv_seq(r, b).ok) dev_report(ctl, DEV_ERR_BAD_BATCH, site);
}

// The sequence that row m belongs to and the row's position, by a whole block at once (one round of
// loads; every thread calls this, once a kernel); b = -1 for a row of no sequence, or of one out of
// range.  Both numbers are one 64-bit word, so that a row that two sequences claim gets one sequence's.
struct KvRow {
  int b, pos;
};
__device__ __forceinline__ KvRow kv_find_row(const KvRows& r, int m) {
  __shared__ unsigned long long at;
  if (threadIdx.x == 0) at = ~0ULL;
  __syncthreads();
  auto claim = [&](int b) {
    const KvSeq s = kv_seq(r, b);  // (the loads of several do not wait for one another)
    const unsigned int i = (unsigned int)m - (unsigned int)s.row0;
    if (i < (unsigned int)s.n) at = (unsigned long long)(s.len - s.n + i) << 32 | (unsigned int)b;
  };
  if (!r.cu) {
    if (threadIdx.x == 0 && m < r.B) claim(m);
  } else {
    for (int b = threadIdx.x; b < r.B; b += blockDim.x) claim(b);
  }
  __syncthreads();
  const unsigned long long v = at;
  return KvRow{(int)(unsigned int)v, (int)(v >> 32)};
}

// Announces `bytes` (a multiple of 16) on the mbarrier at shared address bar and copies them from
// global memory to shared address dst (cp.async.bulk), counted on it.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .b64 st;\n\tmbarrier.arrive.expect_tx.shared::cta.b64 st, [%3], %2;\n\t"
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n\t}" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}
// packed fp32 product (ffma2 and fadd2 are in ptx.cuh)
__device__ __forceinline__ float2 fmul2(float2 a, float2 b) {
  uint64_t d;
  asm("{\n\t.reg .b64 pa, pb;\n\tmov.b64 pa, {%1, %2};\n\tmov.b64 pb, {%3, %4};\n\t"
      "mul.rn.f32x2 %0, pa, pb;\n\t}"
      : "=l"(d)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(d));
  return r;
}

__device__ __forceinline__ float bf16_bits(unsigned int u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf16_lo(unsigned int u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf16_hi(unsigned int u) { return __uint_as_float(u & 0xffff0000u); }

// Host side: checks of the two descriptions every call takes.
int kv_check(const char* what, const gpt_kv_cache* c, const gpt_kv_batch* b, int M);
// Most new tokens of a sequence: one each without cu_new, whatever the field holds.
inline int kv_max_new(const gpt_kv_batch* b) { return b->cu_new ? b->max_new : 1; }
inline KvRows kv_rows(const gpt_kv_batch* b, int M) {
  return KvRows{b->block_table, b->lens, b->cu_new, b->n_seq, b->max_blocks, kv_max_new(b), M};
}

// Calls f(KvGeom<bits, hd>()) for the cache's geometry (kv_check has admitted it).
template <typename F>
int kv_dispatch(const gpt_kv_cache* c, F&& f) {
  if (c->bits == 4) return c->head_dim == 64 ? f(KvGeom<4, 64>()) : f(KvGeom<4, 128>());
  return c->head_dim == 64 ? f(KvGeom<8, 64>()) : f(KvGeom<8, 128>());
}

}  // namespace gptk
