// Writing the quantised key/value cache from raw q|k|v rows, and reading it back.
#include <cfloat>
#include <cmath>
#include <string>

#include "kv.cuh"

namespace gptk {

// ------------------------------------------------------------------ append
//
// One CTA takes the new tokens of one cache block of one sequence (1 .. 64 of them) and a share of
// the heads.  The angles of a token are computed once, in fp64 (position x frequency passes 2^24 on
// long contexts), into shared memory and serve all its heads.  A row (token, head) belongs to HD / 16
// lanes; a lane holds the octets l and l + HD / 16, so both halves of a RoPE pair (d, d + HD / 2) are
// its own.  The warp's 32 / (HD / 16) lane groups take tokens of one head, and the elementwise
// bounds of the block's keys are carried in registers and joined across the groups at the end; a
// block with fewer new tokens than groups (a decoding step) gives each group a head of its own.
struct RopeFreq {
  double f[64];  // base^(-2 i / hd)
};

constexpr int kAppendThreads = 256;

// keeps NaN: a block whose keys hold a NaN has NaN bounds
__device__ __forceinline__ float min_nan(float a, float b) { return (b < a || b != b) ? b : a; }
__device__ __forceinline__ float max_nan(float a, float b) { return (b > a || b != b) ? b : a; }

template <class G>
__global__ void __launch_bounds__(kAppendThreads)
kv_append_kernel(const __nv_bfloat16* __restrict__ qkv, KvRows rows, int blocks_per_seq, uint8_t* __restrict__ tiles,
                 __nv_bfloat16* __restrict__ bounds, int n_blocks, int H, int Hkv, int rope, int qk_norm, float eps,
                 RopeFreq freq, __nv_bfloat16* __restrict__ q_out, DevCtl ctl) {
  constexpr int HD = G::HD, HALF = HD / 2;
  constexpr int LPR = HD / 16;   // lanes of a row
  constexpr int SG = 32 / LPR;   // rows of a warp
  __shared__ float s_cos[kKvBlock][HALF], s_sin[kKvBlock][HALF];
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x / blocks_per_seq;
  const KvSeq s = kv_seq(rows, b);
  if (!s.ok) {
    if (threadIdx.x == 0) dev_report(ctl, DEV_ERR_BAD_BATCH, 1);
    return;
  }
  const int pos0 = s.len - s.n;  // position of the first new token
  const int blk = pos0 / kKvBlock + (blockIdx.x - b * blocks_per_seq);
  const int t0 = max(pos0, blk * kKvBlock), t1 = min(s.len, (blk + 1) * kKvBlock);  // its new tokens
  const int nt = t1 - t0;
  if (nt <= 0) return;
  const int phys = rows.table[(long long)b * rows.W + blk];
  if (phys < 0 || phys >= n_blocks) {
    if (threadIdx.x == 0) dev_report(ctl, DEV_ERR_BAD_BATCH, 2);
    return;
  }
  if (rope) {
    for (int x = threadIdx.x; x < nt * HALF; x += kAppendThreads) {
      const int t = x / HALF, i = x - t * HALF;
      const double a = (double)(t0 + t) * freq.f[i];
      const float red = (float)(a - rint(a * 0.15915494309189535) * 6.283185307179586);
      sincosf(red, &s_sin[t][i], &s_cos[t][i]);
    }
    __syncthreads();
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sg = lane / LPR, l = lane % LPR;
  const bool wide = nt >= SG;       // the groups take tokens of one head; else a head each
  const int heads = H + 2 * Hkv;
  const int hstep = wide ? 1 : SG;  // heads of a warp at a time
  const long long ld = (long long)heads * HD;
  const int warps = gridDim.y * (kAppendThreads / 32);
  for (int h0 = (blockIdx.y * (kAppendThreads / 32) + warp) * hstep; h0 < heads; h0 += warps * hstep) {
    const int h = wide ? h0 : h0 + sg;
    const bool is_k = h >= H && h < H + Hkv, is_v = h >= H + Hkv;
    const int kvh = is_v ? h - H - Hkv : h - H;
    float mn[16], mx[16];
#pragma unroll
    for (int x = 0; x < 16; ++x) mn[x] = INFINITY, mx[x] = -INFINITY;
    for (int tb = 0; tb < nt; tb += wide ? SG : 1) {
      const int t = wide ? tb + sg : tb;
      const bool live = h < heads && t < nt;
      const long long row = s.row0 + (t0 - pos0) + t;
      float a[8], c[8];
      {
        const uint4* p = reinterpret_cast<const uint4*>(qkv + row * ld + (long long)h * HD);
        const uint4 u = live ? __ldg(p + l) : make_uint4(0, 0, 0, 0);
        const uint4 w = live ? __ldg(p + LPR + l) : make_uint4(0, 0, 0, 0);
        const unsigned int uu[4] = {u.x, u.y, u.z, u.w}, ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          a[2 * x] = bf16_lo(uu[x]), a[2 * x + 1] = bf16_hi(uu[x]);
          c[2 * x] = bf16_lo(ww[x]), c[2 * x + 1] = bf16_hi(ww[x]);
        }
      }
      if (qk_norm) {
        float ss = 0.f;
#pragma unroll
        for (int x = 0; x < 8; ++x) ss += a[x] * a[x] + c[x] * c[x];
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float r = is_v ? 1.f : rsqrtf(ss / HD + eps);
#pragma unroll
        for (int x = 0; x < 8; ++x) a[x] *= r, c[x] *= r;
      }
      if (rope && live && !is_v) {
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const float co = s_cos[t][8 * l + x], si = s_sin[t][8 * l + x];
          const float x1 = a[x], x2 = c[x];
          a[x] = x1 * co - x2 * si;
          c[x] = x1 * si + x2 * co;
        }
      }
      if (live && !is_k && !is_v) {
        uint4 u, w;
        unsigned int* uu = &u.x;
        unsigned int* ww = &w.x;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const __nv_bfloat162 pu = __floats2bfloat162_rn(a[2 * x], a[2 * x + 1]);
          const __nv_bfloat162 pw = __floats2bfloat162_rn(c[2 * x], c[2 * x + 1]);
          uu[x] = *reinterpret_cast<const unsigned int*>(&pu);
          ww[x] = *reinterpret_cast<const unsigned int*>(&pw);
        }
        uint4* p = reinterpret_cast<uint4*>(q_out + (row * H + h) * HD);
        p[l] = u;
        p[LPR + l] = w;
      }
      // max |x| of each group as bits, so that an infinity or a NaN is the largest
      unsigned int ma = 0, mc = 0;
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        ma = max(ma, __float_as_uint(a[x]) & 0x7fffffffu);
        mc = max(mc, __float_as_uint(c[x]) & 0x7fffffffu);
      }
      if (G::NG == 1) ma = max(ma, mc);
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) {
        ma = max(ma, __shfl_xor_sync(0xffffffffu, ma, o));
        if (G::NG == 2) mc = max(mc, __shfl_xor_sync(0xffffffffu, mc, o));
      }
      if (G::NG == 1) mc = ma;
      if (live && (is_k || is_v)) {
        // scale = bf16(max / TOP), and the codes are taken against the rounded scale, so its
        // rounding costs no more than the codes' own half step.  A group that holds an infinity or
        // a NaN has a NaN scale; one whose scale would be below the normal range reads as zeros.
        float sf[2];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const unsigned int m = g ? mc : ma;
          float v = __bfloat162float(__float2bfloat16_rn(__fdiv_rn(__uint_as_float(m), (float)G::TOP)));
          if (v < FLT_MIN) v = 0.f;
          if (m >= 0x7f800000u) v = __uint_as_float(0x7fc00000u);
          sf[g] = v;
        }
        const float ia = sf[0] > 0.f ? __fdiv_rn(1.f, sf[0]) : 0.f, ic = sf[1] > 0.f ? __fdiv_rn(1.f, sf[1]) : 0.f;
        int na[8], nc[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          // quotient, then its residual once more: bf16 values over a bf16 scale often lie exactly
          // between two codes, and the bare product with the reciprocal would round those either way
          const float qa = a[x] * ia, qc = c[x] * ic;
          na[x] = min(max(__float2int_rn(fmaf(fmaf(-qa, sf[0], a[x]), ia, qa)), -G::TOP), G::TOP);
          nc[x] = min(max(__float2int_rn(fmaf(fmaf(-qc, sf[1], c[x]), ic, qc)), -G::TOP), G::TOP);
        }
        if (is_k && bounds != nullptr) {
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            const float va = na[x] * sf[0], vc = nc[x] * sf[1];
            mn[x] = min_nan(mn[x], va), mx[x] = max_nan(mx[x], va);
            mn[8 + x] = min_nan(mn[8 + x], vc), mx[8 + x] = max_nan(mx[8 + x], vc);
          }
        }
        const int slot = t0 + t - blk * kKvBlock, i = slot % kKvRec;
        uint8_t* rec = tiles + ((long long)phys * Hkv + kvh) * G::TILE + (slot / kKvRec) * G::REC;
        unsigned int wa[2] = {0, 0}, wc[2] = {0, 0};
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const int at = x * G::BITS;
          wa[at >> 5] |= (unsigned int)(na[x] + G::Z) << (at & 31);
          wc[at >> 5] |= (unsigned int)(nc[x] + G::Z) << (at & 31);
        }
        if (is_k) {
#pragma unroll
          for (int w = 0; w < G::BITS / 4; ++w) {
            *reinterpret_cast<unsigned int*>(rec + G::key_word(i, l * (G::BITS / 4) + w)) = wa[w];
            *reinterpret_cast<unsigned int*>(rec + G::key_word(i, (LPR + l) * (G::BITS / 4) + w)) = wc[w];
          }
        } else if (G::BITS == 4) {
          *reinterpret_cast<unsigned int*>(rec + G::value_octet(i, l)) = wa[0];
          *reinterpret_cast<unsigned int*>(rec + G::value_octet(i, LPR + l)) = wc[0];
        } else {
          *reinterpret_cast<uint2*>(rec + G::value_octet(i, l)) = make_uint2(wa[0], wa[1]);
          *reinterpret_cast<uint2*>(rec + G::value_octet(i, LPR + l)) = make_uint2(wc[0], wc[1]);
        }
        if (l < G::NG) {
          __nv_bfloat16* sp = reinterpret_cast<__nv_bfloat16*>(rec + (is_k ? G::KSCALE : G::VSCALE));
          sp[i * G::NG + l] = __float2bfloat16_rn(l == 0 ? sf[0] : sf[1]);
        }
      }
    }
    if (bounds != nullptr && __any_sync(0xffffffffu, is_k)) {
      if (wide) {
#pragma unroll
        for (int o = LPR; o < 32; o <<= 1) {
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            mn[x] = min_nan(mn[x], __shfl_xor_sync(0xffffffffu, mn[x], o));
            mx[x] = max_nan(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], o));
          }
        }
      }
      if (is_k && (!wide || sg == 0)) {
        const bool join = t0 > blk * kKvBlock;  // tokens of earlier calls are in the block
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          __nv_bfloat16* bp = bounds + (((long long)phys * Hkv + kvh) * 2 + q) * HD;
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            uint4* p = reinterpret_cast<uint4*>(bp) + l + hf * LPR;
            uint4 u = join ? *p : make_uint4(0, 0, 0, 0);
            unsigned int* uu = &u.x;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              float v[2];
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const float old = y ? bf16_hi(uu[x]) : bf16_lo(uu[x]);
                const float w = (q ? mx : mn)[8 * hf + 2 * x + y];
                v[y] = !join ? w : q ? max_nan(old, w) : min_nan(old, w);
              }
              // rounded outward, so that they stay bounds
              const __nv_bfloat16 e0 = q ? __float2bfloat16_ru(v[0]) : __float2bfloat16_rd(v[0]);
              const __nv_bfloat16 e1 = q ? __float2bfloat16_ru(v[1]) : __float2bfloat16_rd(v[1]);
              uu[x] = (unsigned int)__bfloat16_as_ushort(e0) | ((unsigned int)__bfloat16_as_ushort(e1) << 16);
            }
            *p = u;
          }
        }
      }
    }
  }
}

// ------------------------------------------------------------------ read
//
// One warp takes 16 tokens of one kv head: the same 8- or 16-byte pieces per lane that the attention
// kernel reads, straight from global memory, each turned into rows of bf16 values (64 to 128
// contiguous bytes a store instruction and token).
template <class G>
__global__ void __launch_bounds__(256)
kv_read_kernel(KvRows rows, int tiles_per_seq, const uint8_t* __restrict__ tiles, int n_blocks, int Hkv,
               __nv_bfloat16* __restrict__ k_out, __nv_bfloat16* __restrict__ v_out, DevCtl ctl) {
  constexpr int HD = G::HD;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
  const long long total = (long long)rows.B * tiles_per_seq * Hkv;
  const long long step = (long long)gridDim.x * 8;
  for (long long w = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); w < total; w += step) {
    const int h = (int)(w % Hkv);
    const long long bt = w / Hkv;
    const int b = (int)(bt / tiles_per_seq);
    const KvSeq s = kv_seq(rows, b);
    if (!s.ok) {
      if (lane == 0) dev_report(ctl, DEV_ERR_BAD_BATCH, 3);
      continue;
    }
    const int pos0 = s.len - s.n;
    const int tile = pos0 / 16 + (int)(bt - (long long)b * tiles_per_seq);  // 16-token tile of the sequence
    const int base = tile * 16;
    if (base >= s.len) continue;
    const int phys = rows.table[(long long)b * rows.W + base / kKvBlock];
    const bool bad = phys < 0 || phys >= n_blocks;
    if (bad && lane == 0) dev_report(ctl, DEV_ERR_BAD_BATCH, 4);
    const int slot = base % kKvBlock, i0 = slot % kKvRec;
    const uint8_t* rec = tiles + ((long long)(bad ? 0 : phys) * Hkv + h) * G::TILE + (slot / kKvRec) * G::REC;
    const long long row_of = (long long)s.row0 - pos0 + base;  // row of the tile's first token
    auto live = [&](int i) { return base + i >= pos0 && base + i < s.len; };
    auto scale = [&](int off, int i, int g) {
      const unsigned short u = __ldg(reinterpret_cast<const unsigned short*>(rec + off) + (i0 + i) * G::NG + g);
      return bad ? __uint_as_float(0x7fc00000u) : bf16_bits(u);
    };
    auto put = [&](__nv_bfloat16* out, const unsigned int* words, float sf) {  // 8 dims
      uint4 o;
      unsigned int* oo = &o.x;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int at = 2 * x * G::BITS;
        const unsigned int two = words[at >> 5] >> (at & 31);
        const float v0 = sf * (float)((int)(two & (2 * G::Z - 1)) - G::Z);
        const float v1 = sf * (float)((int)((two >> G::BITS) & (2 * G::Z - 1)) - G::Z);
        const __nv_bfloat162 p = __floats2bfloat162_rn(v0, v1);
        oo[x] = *reinterpret_cast<const unsigned int*>(&p);
      }
      *reinterpret_cast<uint4*>(out) = o;
    };
    // values: four keys of this lane, VB bytes each
    {
      unsigned int u[G::VB];  // 4 VB bytes
#pragma unroll
      for (int p = 0; p < G::VB / 4; ++p) {
        const uint4 x = __ldg(reinterpret_cast<const uint4*>(rec + G::VCODES + i0 * G::ROWB + p * 512 + lane * 16));
        u[4 * p] = x.x, u[4 * p + 1] = x.y, u[4 * p + 2] = x.z, u[4 * p + 3] = x.w;
      }
#pragma unroll
      for (int sl = 0; sl < 4; ++sl) {
        const int i = 2 * c + (sl & 1) + 8 * (sl >> 1);
        if (live(i)) {
          __nv_bfloat16* out = v_out + ((row_of + i) * Hkv + h) * HD;
#pragma unroll
          for (int wj = 0; wj < HD / 64; ++wj)
            put(out + 64 * wj + 8 * r, u + (sl * G::VB + wj * G::BITS) / 4, scale(G::VSCALE, i, G::NG == 1 ? 0 : wj));
        }
      }
    }
    // keys: rows r and r + 8 of this lane, KB bytes each: words c, c + 4, ...
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const int i = r + 8 * hf;
      unsigned int u[G::KB / 4];
#pragma unroll
      for (int p = 0; p < G::KB / G::KP; ++p) {
        const uint8_t* at = rec + i0 * G::ROWB + p * 64 * G::KP + i * 4 * G::KP + c * G::KP;
        if (G::KP == 16) {
          const uint4 x = __ldg(reinterpret_cast<const uint4*>(at));
          u[4 * p] = x.x, u[4 * p + 1] = x.y, u[4 * p + 2] = x.z, u[4 * p + 3] = x.w;
        } else {
          const uint2 x = __ldg(reinterpret_cast<const uint2*>(at));
          u[0] = x.x, u[1] = x.y;
        }
      }
      if (live(i)) {
        __nv_bfloat16* out = k_out + ((row_of + i) * Hkv + h) * HD;
        if (G::BITS == 4) {
#pragma unroll
          for (int wi = 0; wi < G::KB / 4; ++wi)
            put(out + 32 * wi + 8 * c, u + wi, scale(G::KSCALE, i, G::NG == 1 ? 0 : wi / 2));
        } else {
          const float sf = scale(G::KSCALE, i, 0);
#pragma unroll
          for (int wi = 0; wi < G::KB / 4; ++wi) {
            uint2 o;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const float v0 = sf * (float)((int)((u[wi] >> (16 * x)) & 255) - G::Z);
              const float v1 = sf * (float)((int)((u[wi] >> (16 * x + 8)) & 255) - G::Z);
              const __nv_bfloat162 p = __floats2bfloat162_rn(v0, v1);
              (x ? o.y : o.x) = *reinterpret_cast<const unsigned int*>(&p);
            }
            *reinterpret_cast<uint2*>(out + 16 * wi + 4 * c) = o;
          }
        }
      }
    }
  }
}

// ------------------------------------------------------------------ host

static bool misaligned(const void* p, unsigned int to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

int kv_check(const char* what, const gpt_kv_cache* c, const gpt_kv_batch* b, int M) {
  const std::string w(what);
  if (!c || !b) return set_error(ST_INVALID_ARG, w + ": null cache or batch");
  if (c->bits != 4 && c->bits != 8) return set_error(ST_UNSUPPORTED, w + ": the cache holds 4 or 8 bits");
  if (c->head_dim != 64 && c->head_dim != 128) return set_error(ST_UNSUPPORTED, w + ": head dim must be 64 or 128");
  if (c->n_blocks < 1 || c->n_kv_head < 1) return set_error(ST_INVALID_ARG, w + ": n_blocks and n_kv_head must be >= 1");
  if (!c->tiles) return set_error(ST_INVALID_ARG, w + ": null tiles");
  if (misaligned(c->tiles, 16) || misaligned(c->bounds, 16))
    return set_error(ST_INVALID_ARG, w + ": tiles and bounds must be 16-byte aligned");
  if (b->n_seq < 0 || b->max_blocks < 1 || b->max_new < 0)
    return set_error(ST_INVALID_ARG, w + ": n_seq and max_new must be >= 0, max_blocks >= 1");
  if (M < 0) return set_error(ST_INVALID_ARG, w + ": M must be >= 0");
  if (b->max_blocks > (1 << 24)) return set_error(ST_UNSUPPORTED, w + ": max_blocks above 2^24");
  if (b->n_seq > 0 && (!b->block_table || !b->lens)) return set_error(ST_INVALID_ARG, w + ": null block_table or lens");
  if (!b->cu_new && b->n_seq > M)
    return set_error(ST_INVALID_ARG, w + ": without cu_new every sequence has one row: M must be >= n_seq");
  if (misaligned(b->block_table, 4) || misaligned(b->lens, 4) || misaligned(b->cu_new, 4))
    return set_error(ST_INVALID_ARG, w + ": block_table, lens and cu_new must be 4-byte aligned");
  return ST_OK;
}

}  // namespace gptk

using namespace gptk;

extern "C" {

GPT_API int gpt_kv_tile_bytes(int bits, int head_dim, size_t* bytes) {
  set_error(ST_OK, "");
  if (!bytes) return set_error(ST_INVALID_ARG, "kv_tile_bytes: null output");
  if (bits != 4 && bits != 8) return set_error(ST_UNSUPPORTED, "kv_tile_bytes: the cache holds 4 or 8 bits");
  if (head_dim != 64 && head_dim != 128) return set_error(ST_UNSUPPORTED, "kv_tile_bytes: head dim must be 64 or 128");
  gpt_kv_cache c = {};
  c.bits = bits;
  c.head_dim = head_dim;
  return kv_dispatch(&c, [&](auto g) {
    *bytes = decltype(g)::TILE;
    return (int)ST_OK;
  });
}

GPT_API int gpt_op_kv_append(const gpt_kv_cache* cache, const gpt_kv_batch* batch, const void* qkv, int M, int H,
                             int rope, int qk_norm, float rope_base, float eps, void* q_out, void* stream) {
  set_error(ST_OK, "");
  GPTK_TRY(kv_check("kv_append", cache, batch, M));
  const int Hkv = cache->n_kv_head;
  if (H < 1 || H % Hkv) return set_error(ST_INVALID_ARG, "kv_append: H must be a multiple of n_kv_head");
  if ((long long)H + 2LL * Hkv > 65536) return set_error(ST_UNSUPPORTED, "kv_append: more than 65536 heads");
  if (rope && !(rope_base > 1.f)) return set_error(ST_INVALID_ARG, "kv_append: rope_base must be > 1");
  if (qk_norm && !(eps > 0.f)) return set_error(ST_INVALID_ARG, "kv_append: eps must be > 0");
  if (M == 0 || batch->n_seq == 0 || batch->max_new == 0) return ST_OK;
  if (!qkv || !q_out) return set_error(ST_INVALID_ARG, "kv_append: null qkv or q_out");
  if (misaligned(qkv, 16) || misaligned(q_out, 16))
    return set_error(ST_INVALID_ARG, "kv_append: qkv and q_out must be 16-byte aligned");
  const int max_new = batch->cu_new ? batch->max_new : 1;
  const long long bps = ((long long)max_new + kKvBlock - 2) / kKvBlock + 1;  // blocks that max_new tokens can touch
  if (bps * batch->n_seq > 0x7fffffffLL) return set_error(ST_UNSUPPORTED, "kv_append: n_seq x max_new too large");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  RopeFreq f;
  for (int i = 0; i < 64; ++i)
    f.f[i] = rope ? std::pow((double)rope_base, -2.0 * i / cache->head_dim) : 0.0;
  const double row = (double)(H + 2 * Hkv) * cache->head_dim;
  Prof prof(PK_QK, 0, M * row * 2 + (double)M * H * cache->head_dim * 2, st);
  return kv_dispatch(cache, [&](auto g) -> int {
    using G = decltype(g);
    // the heads are shared among enough CTAs to give every SM a few
    const long long ctas = bps * batch->n_seq;
    const int hw = max_new >= 8 ? H + 2 * Hkv : (H + 2 * Hkv + 3) / 4;
    long long y = ctas >= 4LL * num_sms() ? 1 : (4LL * num_sms() + ctas - 1) / ctas;
    if (y > (hw + 7) / 8) y = (hw + 7) / 8;
    KvRows r = kv_rows(batch, M);
    r.max_new = max_new;
    GPTK_CUDA(launch_pdl(kv_append_kernel<G>, dim3((unsigned)ctas, (unsigned)y), dim3(kAppendThreads), 0, st,
                         static_cast<const __nv_bfloat16*>(qkv), r, (int)bps, static_cast<uint8_t*>(cache->tiles),
                         static_cast<__nv_bfloat16*>(cache->bounds), (int)cache->n_blocks, H, Hkv, rope, qk_norm, eps, f,
                         static_cast<__nv_bfloat16*>(q_out), device_ctl()));
    return ST_OK;
  });
}

GPT_API int gpt_op_kv_read(const gpt_kv_cache* cache, const gpt_kv_batch* batch, int M, void* k_out, void* v_out,
                           void* stream) {
  set_error(ST_OK, "");
  GPTK_TRY(kv_check("kv_read", cache, batch, M));
  if (M == 0 || batch->n_seq == 0 || batch->max_new == 0) return ST_OK;
  if (!k_out || !v_out) return set_error(ST_INVALID_ARG, "kv_read: null k_out or v_out");
  if (misaligned(k_out, 16) || misaligned(v_out, 16))
    return set_error(ST_INVALID_ARG, "kv_read: k_out and v_out must be 16-byte aligned");
  const int Hkv = cache->n_kv_head;
  const int max_new = batch->cu_new ? batch->max_new : 1;
  const long long tps = ((long long)max_new + 14) / 16 + 1;  // 16-token tiles that max_new tokens can touch
  if (tps > 0x7fffffffLL) return set_error(ST_UNSUPPORTED, "kv_read: max_new too large");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  Prof prof(PK_MISC, 0, (double)M * Hkv * cache->head_dim * (4 + cache->bits / 4.0), st);
  return kv_dispatch(cache, [&](auto g) -> int {
    using G = decltype(g);
    const long long items = tps * batch->n_seq * Hkv;
    const long long want = (items + 7) / 8, most = 8LL * num_sms();
    KvRows r = kv_rows(batch, M);
    r.max_new = max_new;
    GPTK_CUDA(launch_pdl(kv_read_kernel<G>, dim3((unsigned)(want < most ? want : most)), dim3(256), 0, st, r, (int)tps,
                         static_cast<const uint8_t*>(cache->tiles), (int)cache->n_blocks, Hkv,
                         static_cast<__nv_bfloat16*>(k_out), static_cast<__nv_bfloat16*>(v_out), device_ctl()));
    return ST_OK;
  });
}

}  // extern "C"
