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
// Bounded by latency with four warps a scheduler: 18.5k tokens of 30 heads of 128 in 4 bits take 58 us (33 of
// bytes), 3.7 TB/s, at 0.61 instructions a clock and scheduler; for each, a warp waits 1.35 issue slots for its own
// results and 0.9 for shared memory, the ring's and the tables' (a third CTA an SM would spill: 70 us).  A step of 16
// tokens takes 3 us.
struct RopeFreq {
  double f[64];  // base^(-2 i / hd)
};

constexpr int kAppendThreads = 256;

// keeps NaN: a block whose keys hold a NaN has NaN bounds
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Eight values of one scale group to codes.  x / s is the product with an approximate reciprocal plus
// its residual once more (Markstein's correction of an approximate quotient by fused multiply-adds, 1990), which
// is exact where fp32 holds the quotient: bf16 values over a bf16 scale often
// lie exactly between two codes, and the bare product would round those either way.  Adding 1.5 2^23 + Z
// rounds it to the integer code in the sum's low bits (one fp32 add; a float-to-int conversion has an
// eighth of its rate).  |x / s| <= top (1 + 2^-8) rounds to at most top, so nothing is clamped.
template <class G>
struct Coded {
  unsigned int w[G::BITS / 4];  // code words of the eight dims
  float2 n[4];                  // code - Z as floats
};
template <class G>
__device__ __forceinline__ Coded<G> encode8(const float2 (&x)[4], float s, float inv) {
  Coded<G> r;
  constexpr float MAGIC = 12582912.f + G::Z;
  const float2 ns = make_float2(-s, -s), i2 = make_float2(inv, inv), mg = make_float2(MAGIC, MAGIC);
  unsigned int t[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 q = fmul2(x[i], i2);
    const float2 f = fadd2(ffma2(ffma2(q, ns, x[i]), i2, q), mg);
    r.n[i] = fadd2(f, make_float2(-MAGIC, -MAGIC));
    t[2 * i] = __float_as_uint(f.x), t[2 * i + 1] = __float_as_uint(f.y);
  }
  // the low bytes, four to a word
  auto bytes = [](unsigned int b0, unsigned int b1, unsigned int b2, unsigned int b3) {
    return __byte_perm(__byte_perm(b0, b1, 0x0040), __byte_perm(b2, b3, 0x0040), 0x5410);
  };
  if (G::BITS == 8) {
    r.w[0] = bytes(t[0], t[1], t[2], t[3]);
    r.w[G::BITS / 4 - 1] = bytes(t[4], t[5], t[6], t[7]);
  } else {
    r.w[0] = (bytes(t[0], t[2], t[4], t[6]) & 0x0f0f0f0fu) + ((bytes(t[1], t[3], t[5], t[7]) & 0x0f0f0f0fu) << 4);
  }
  return r;
}

// cos and sin of an angle of any size: reduced in fp64 to r in [-pi/4, pi/4] and a quarter turn k (adding
// 1.5 2^52 rounds to the integer, whose low bits it leaves in the sum's low word), then the Taylor sums to
// r^9 and r^10 in fp32, whose remainders (1.8e-9 and 1.2e-10 at pi/4) are below fp32's rounding.  The
// arguments reach pi/4 only, so this takes a third of the instructions of the general functions.
__device__ __forceinline__ void rope_angle(double a, float* c, float* s) {
  constexpr double kShift = 6755399441055744.0;  // 1.5 2^52
  const double t = fma(a, 0.6366197723675814, kShift);
  const int k = __double2loint(t);
  const float r = (float)fma(kShift - t, 1.5707963267948966, a), z = r * r;
  float sn = fmaf(z, 1.f / 362880.f, -1.f / 5040.f);
  sn = fmaf(sn, z, 1.f / 120.f);
  sn = fmaf(sn, z, -1.f / 6.f);
  sn = fmaf(sn * z, r, r);
  float cs = fmaf(z, -1.f / 3628800.f, 1.f / 40320.f);
  cs = fmaf(cs, z, -1.f / 720.f);
  cs = fmaf(cs, z, 1.f / 24.f);
  cs = fmaf(cs, z, -0.5f);
  cs = fmaf(cs, z, 1.f);
  const bool odd = k & 1;
  const float x = odd ? sn : cs, y = odd ? cs : sn;
  *c = (k + 1) & 2 ? -x : x;
  *s = k & 2 ? -y : y;
}

// The raw rows come through a ring of asynchronous copies, private to each lane: it reads back the 32
// bytes a turn that it copied itself, so the ring needs no barrier.  Three turns in flight by 16 warps
// are 48 KB an SM, what HBM's latency asks for; loads into registers one turn ahead were a third of that
// and bounded the kernel (63 us against 58 for 18.5k tokens of 30 heads).
constexpr int kAppendRing = 4;
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// What a CTA of the append has in hand for all of its heads.
struct AppendCta {
  const __nv_bfloat16* src;  // raw row of the block's first new token, at this lane's octet
  __nv_bfloat16* q_out;      // q row of that token, at this lane's octet
  uint8_t* tiles;            // of the cache block
  __nv_bfloat16* bounds;     // of the cache block, or null
  const float4 *cos, *sin;   // of the first new token, at this lane's first piece
  long long ld;              // raw row pitch
  int H, Hkv, nt, slot0, sg, l;
  bool rope, norm, join;     // join: the block holds tokens of earlier calls
  float eps;
  // the copying iterator: head step, token turn, and the shared address of this lane's ring
  int f_h, f_tb, heads, hs;
  bool wide;
  uint32_t ring;
  int turn;                  // turns read so far
};

// Starts the copy of the next turn's item (head f_h, or f_h + sg; token f_tb + sg, or f_tb) into the slot
// of turn `turn`, if there is one; a group either way, so that the waits can count.
template <class G>
__device__ __forceinline__ void append_copy(AppendCta& c, int turn) {
  constexpr int LPR = G::HD / 16, SG = 32 / LPR;
  if (c.f_h < c.heads) {
    const int h = c.wide ? c.f_h : c.f_h + c.sg, t = c.wide ? c.f_tb + c.sg : c.f_tb;
    const bool live = h < c.heads && t < c.nt;
    const __nv_bfloat16* p = c.src + (live ? t * c.ld + (long long)h * G::HD : 0);
    const uint32_t dst = c.ring + turn % kAppendRing * 1024;
    copy16(dst, p, live);
    copy16(dst + 512, p + 8 * LPR, live);
    c.f_tb += c.wide ? SG : 1;
    if (c.f_tb >= c.nt) c.f_tb = 0, c.f_h += c.hs;
  }
  copy_commit();
}

enum { kRowQ, kRowK, kRowV, kRowMixed };

// The tokens of one head (KIND q, k or v: the warp's lane groups take tokens), or of a head for each
// lane group (kRowMixed).
template <class G, int KIND>
__device__ __forceinline__ void append_head(AppendCta& a_, int h, bool in_range) {
  constexpr int HD = G::HD, HALF = HD / 2, LPR = HD / 16, SG = 32 / LPR;
  constexpr bool MIXED = KIND == kRowMixed;
  constexpr int NW = G::BITS / 4;  // code words of an octet
  const int H = a_.H, Hkv = a_.Hkv, nt = a_.nt, l = a_.l;
  const bool is_k = MIXED ? h >= H && h < H + Hkv : KIND == kRowK;
  const bool is_v = MIXED ? h >= H + Hkv : KIND == kRowV;
  const bool is_q = !is_k && !is_v;
  const int tstep = MIXED ? 1 : SG;
  uint8_t* tile = a_.tiles + (long long)(is_v ? h - H - Hkv : is_k ? h - H : 0) * G::TILE;
  // a code word's place is a token's offset plus a lane's (key_word and value_octet are sums of both)
  int off_a, off_c;
  if (is_v) off_a = G::value_octet(0, l), off_c = G::value_octet(0, LPR + l);
  else off_a = G::key_word(0, l * NW), off_c = G::key_word(0, (LPR + l) * NW);
  float mn[16], mx[16];
  if (KIND == kRowK || MIXED) {
#pragma unroll
    for (int x = 0; x < 16; ++x) mn[x] = INFINITY, mx[x] = -INFINITY;
  }
  for (int t = MIXED ? 0 : a_.sg, tb = 0; tb < nt; tb += tstep, t += tstep) {
    const bool live = in_range && t < nt;
    float2 a[4], c[4];
    {
      copy_wait<kAppendRing - 2>();
      unsigned int uu[4], ww[4];
      const uint32_t at = a_.ring + a_.turn % kAppendRing * 1024;
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(uu[0]), "=r"(uu[1]), "=r"(uu[2]), "=r"(uu[3])
                   : "r"(at)
                   : "memory");
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(ww[0]), "=r"(ww[1]), "=r"(ww[2]), "=r"(ww[3])
                   : "r"(at + 512)
                   : "memory");
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        a[x] = make_float2(bf16_lo(uu[x]), bf16_hi(uu[x]));
        c[x] = make_float2(bf16_lo(ww[x]), bf16_hi(ww[x]));
      }
      append_copy<G>(a_, a_.turn + kAppendRing - 1);  // the slot of the turn before, which has been read
      ++a_.turn;
    }
    // The norm's factor r = rsqrt(mean x^2 + eps) scales a whole row, so RoPE and the largest value
    // are taken on the raw row (max |r x| = r max |x|) and the reductions of both run together.
    float ss = 0.f, ma = 0.f, mc = 0.f;  // sum of squares; max |x| of each group, a NaN stays
    if (KIND != kRowV && a_.norm) {
      float2 s2 = fmul2(a[0], a[0]);
#pragma unroll
      for (int x = 1; x < 4; ++x) s2 = ffma2(a[x], a[x], s2);
#pragma unroll
      for (int x = 0; x < 4; ++x) s2 = ffma2(c[x], c[x], s2);
      ss = s2.x + s2.y;
    }
    if (KIND != kRowV && a_.rope && live && !is_v) {
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const float4 co = a_.cos[t * (HALF / 4) + y * LPR], si = a_.sin[t * (HALF / 4) + y * LPR];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float2 co2 = x ? make_float2(co.z, co.w) : make_float2(co.x, co.y);
          const float2 si2 = x ? make_float2(si.z, si.w) : make_float2(si.x, si.y);
          const float2 x1 = a[2 * y + x], x2 = c[2 * y + x];
          a[2 * y + x] = ffma2(x1, co2, fmul2(x2, make_float2(-si2.x, -si2.y)));
          c[2 * y + x] = ffma2(x1, si2, fmul2(x2, co2));
        }
      }
    }
    if (KIND != kRowQ) {
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        ma = max_nan(max_nan(ma, fabsf(a[x].x)), fabsf(a[x].y));
        mc = max_nan(max_nan(mc, fabsf(c[x].x)), fabsf(c[x].y));
      }
      if (G::NG == 1) ma = max_nan(ma, mc);
    }
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) {
      if (KIND != kRowV) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (KIND != kRowQ) ma = max_nan(ma, __shfl_xor_sync(0xffffffffu, ma, o));
      if (KIND != kRowQ && G::NG == 2) mc = max_nan(mc, __shfl_xor_sync(0xffffffffu, mc, o));
    }
    if (KIND != kRowV && a_.norm) {
      const float r = is_v ? 1.f : rsqrtf(ss / HD + a_.eps);
      const float2 r2 = make_float2(r, r);
      ma *= r, mc *= r;
#pragma unroll
      for (int x = 0; x < 4; ++x) a[x] = fmul2(a[x], r2), c[x] = fmul2(c[x], r2);
    }
    if (G::NG == 1) mc = ma;
    if ((KIND == kRowQ || MIXED) && live && is_q) {
      uint4 ou, ow;
      unsigned int* uu = &ou.x;
      unsigned int* ww = &ow.x;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const __nv_bfloat162 pu = __floats2bfloat162_rn(a[x].x, a[x].y);
        const __nv_bfloat162 pw = __floats2bfloat162_rn(c[x].x, c[x].y);
        uu[x] = *reinterpret_cast<const unsigned int*>(&pu);
        ww[x] = *reinterpret_cast<const unsigned int*>(&pw);
      }
      uint4* p = reinterpret_cast<uint4*>(a_.q_out + ((long long)t * H + h) * HD);
      p[0] = ou;
      p[LPR] = ow;
    }
    if (KIND != kRowQ && live && !is_q) {
      // scale = bf16(max / TOP), and the codes are taken against the rounded scale, so its
      // rounding costs no more than the codes' own half step.  A group that holds an infinity or
      // a NaN has a NaN scale; one whose scale would be below the normal range reads as zeros.
      float sf[2], inv[2];
#pragma unroll
      for (int g = 0; g < G::NG; ++g) {
        const float m = g ? mc : ma;
        constexpr float RT = 1.f / G::TOP;
        const float q = m * RT;  // and its residual, as in encode8: m / TOP correctly rounded
        float v = __bfloat162float(__float2bfloat16_rn(fmaf(fmaf(-q, (float)G::TOP, m), RT, q)));
        if (v < FLT_MIN) v = 0.f;
        if (!(m < INFINITY)) v = __uint_as_float(0x7fc00000u);
        sf[g] = v;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv[g]) : "f"(v));
        if (v == 0.f) inv[g] = 0.f;
      }
      if (G::NG == 1) sf[1] = sf[0], inv[1] = inv[0];
      const Coded<G> ca = encode8<G>(a, sf[0], inv[0]), cc = encode8<G>(c, sf[1], inv[1]);
      if ((KIND == kRowK || MIXED) && is_k && a_.bounds != nullptr) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float2 va = fmul2(ca.n[x], make_float2(sf[0], sf[0])), vc = fmul2(cc.n[x], make_float2(sf[1], sf[1]));
          mn[2 * x] = min_nan(mn[2 * x], va.x), mx[2 * x] = max_nan(mx[2 * x], va.x);
          mn[2 * x + 1] = min_nan(mn[2 * x + 1], va.y), mx[2 * x + 1] = max_nan(mx[2 * x + 1], va.y);
          mn[8 + 2 * x] = min_nan(mn[8 + 2 * x], vc.x), mx[8 + 2 * x] = max_nan(mx[8 + 2 * x], vc.x);
          mn[9 + 2 * x] = min_nan(mn[9 + 2 * x], vc.y), mx[9 + 2 * x] = max_nan(mx[9 + 2 * x], vc.y);
        }
      }
      const int slot = a_.slot0 + t, i = slot % kKvRec;
      uint8_t* rec = tile + slot / kKvRec * G::REC;
      uint8_t* at = rec + (is_v ? G::value_octet(i, 0) - G::VCODES : G::key_word(i, 0));
      if (is_v && NW == 2) {
        *reinterpret_cast<uint2*>(at + off_a) = make_uint2(ca.w[0], ca.w[NW - 1]);
        *reinterpret_cast<uint2*>(at + off_c) = make_uint2(cc.w[0], cc.w[NW - 1]);
      } else {  // the two words of an 8-bit key octet belong to neighbouring lanes' pieces
        *reinterpret_cast<unsigned int*>(at + off_a) = ca.w[0];
        *reinterpret_cast<unsigned int*>(at + off_c) = cc.w[0];
        if (NW == 2) {
          *reinterpret_cast<unsigned int*>(at + off_a + G::KP) = ca.w[NW - 1];
          *reinterpret_cast<unsigned int*>(at + off_c + G::KP) = cc.w[NW - 1];
        }
      }
      if (l < G::NG) {
        __nv_bfloat16* sp = reinterpret_cast<__nv_bfloat16*>(rec + (is_v ? G::VSCALE : G::KSCALE));
        sp[i * G::NG + l] = __float2bfloat16_rn(l == 0 ? sf[0] : sf[1]);
      }
    }
  }
  if ((KIND == kRowK || MIXED) && a_.bounds != nullptr && (!MIXED || __any_sync(0xffffffffu, is_k))) {
    if (!MIXED) {
#pragma unroll
      for (int o = LPR; o < 32; o <<= 1) {
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          mn[x] = min_nan(mn[x], __shfl_xor_sync(0xffffffffu, mn[x], o));
          mx[x] = max_nan(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], o));
        }
      }
    }
    if (is_k && in_range && (MIXED || a_.sg == 0)) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        __nv_bfloat16* bp = a_.bounds + ((h - H) * 2LL + q) * HD;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint4* p = reinterpret_cast<uint4*>(bp) + l + hf * LPR;
          uint4 bu = a_.join ? *p : make_uint4(0, 0, 0, 0);
          unsigned int* uu = &bu.x;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            float v[2];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const float old = y ? bf16_hi(uu[x]) : bf16_lo(uu[x]);
              const float f = (q ? mx : mn)[8 * hf + 2 * x + y];
              v[y] = !a_.join ? f : q ? max_nan(old, f) : min_nan(old, f);
            }
            // rounded outward, so that they stay bounds
            const __nv_bfloat16 e0 = q ? __float2bfloat16_ru(v[0]) : __float2bfloat16_rd(v[0]);
            const __nv_bfloat16 e1 = q ? __float2bfloat16_ru(v[1]) : __float2bfloat16_rd(v[1]);
            uu[x] = (unsigned int)__bfloat16_as_ushort(e0) | ((unsigned int)__bfloat16_as_ushort(e1) << 16);
          }
          *p = bu;
        }
      }
    }
  }
}

template <class G>
__global__ void __launch_bounds__(kAppendThreads)
kv_append_kernel(const __nv_bfloat16* __restrict__ qkv, KvRows rows, int blocks_per_seq, uint8_t* __restrict__ tiles,
                 __nv_bfloat16* __restrict__ bounds, int n_blocks, int H, int Hkv, int rope, int qk_norm, float eps,
                 RopeFreq freq, __nv_bfloat16* __restrict__ q_out, DevCtl ctl) {
  constexpr int HD = G::HD, HALF = HD / 2;
  constexpr int LPR = HD / 16;   // lanes of a row
  constexpr int SG = 32 / LPR;   // rows of a warp
  // cosines and sines of a token's frequencies, in pieces of four: piece y of lane l (frequencies
  // 8 l + 4 y ..) at y LPR + l, so that a read takes consecutive pieces
  extern __shared__ __align__(128) uint8_t append_smem[];
  float4(*s_cos)[HALF / 4] = reinterpret_cast<float4(*)[HALF / 4]>(append_smem);
  float4(*s_sin)[HALF / 4] = s_cos + kKvBlock;
  uint8_t* s_ring = append_smem + 2 * kKvBlock * HALF * 4;
  pdl_wait();
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
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sg = lane / LPR, l = lane % LPR;
  const bool wide = nt >= SG;       // the lane groups take tokens of one head; else a head each
  const int heads = H + 2 * Hkv;
  const int hstep = wide ? 1 : SG;  // heads of a warp at a time
  const long long row = s.row0 + (t0 - pos0);
  AppendCta c;
  c.ld = (long long)heads * HD;
  c.src = qkv + row * c.ld + 8 * l;
  c.q_out = q_out + row * H * HD + 8 * l;
  c.tiles = tiles + (long long)phys * Hkv * G::TILE;
  c.bounds = bounds ? bounds + (long long)phys * Hkv * 2 * HD : nullptr;
  c.cos = &s_cos[0][l], c.sin = &s_sin[0][l];
  c.H = H, c.Hkv = Hkv, c.nt = nt, c.slot0 = t0 - blk * kKvBlock, c.sg = sg, c.l = l;
  c.rope = rope, c.norm = qk_norm, c.join = c.slot0 > 0, c.eps = eps;
  const int hs = gridDim.y * (kAppendThreads / 32) * hstep;
  int h0 = (blockIdx.y * (kAppendThreads / 32) + warp) * hstep;
  c.heads = heads, c.hs = hs, c.wide = wide, c.f_h = h0, c.f_tb = 0, c.turn = 0;
  c.ring = smem_u32(s_ring) + warp * kAppendRing * 1024 + lane * 16;
#pragma unroll
  for (int i = 0; i < kAppendRing - 1; ++i) append_copy<G>(c, i);
  if (rope) {
    float* fc = reinterpret_cast<float*>(s_cos);
    float* fs = reinterpret_cast<float*>(s_sin);
    for (int x = threadIdx.x; x < nt * HALF; x += kAppendThreads) {
      const int t = x / HALF, at = x - t * HALF;
      const int i = at / 4 % LPR * 8 + at / 4 / LPR * 4 + at % 4;
      rope_angle((double)(t0 + t) * freq.f[i], fc + x, fs + x);
    }
    __syncthreads();
  }
  for (; h0 < heads; h0 += hs) {
    if (!wide) append_head<G, kRowMixed>(c, h0 + sg, h0 + sg < heads);
    else if (h0 < H) append_head<G, kRowQ>(c, h0, true);
    else if (h0 < H + Hkv) append_head<G, kRowK>(c, h0, true);
    else append_head<G, kRowV>(c, h0, true);
  }
  copy_wait<0>();
}

// ------------------------------------------------------------------ read
//
// One CTA takes a cache block of a sequence, one warp a kv head, 16 tokens at a time: the same 8- or
// 16-byte pieces per lane that the attention kernel reads, straight from global memory, each turned
// into rows of bf16 values (64 to 128 contiguous bytes a store instruction and token).  A code becomes
// a float by setting it into the low bits of 2^23.  Bounded by HBM, mostly writes: 28k tokens of 13 heads of
// 128 in 8 bits take 54.5 us, 5.2 TB/s; one sequence of 777 tokens 7 us, launch and three dependent loads.
template <class G>
__global__ void __launch_bounds__(256)
kv_read_kernel(KvRows rows, int blocks_per_seq, const uint8_t* tiles, int n_blocks, int Hkv,
               __nv_bfloat16* k_out, __nv_bfloat16* v_out, DevCtl ctl) {
  constexpr int HD = G::HD;
  const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
  const int h = blockIdx.y * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int b = blockIdx.x / blocks_per_seq;
  pdl_wait();
  if (h >= Hkv) return;
  const KvSeq s = kv_seq(rows, b);
  if (!s.ok) {
    if (lane == 0) dev_report(ctl, DEV_ERR_BAD_BATCH, 3);
    return;
  }
  const int pos0 = s.len - s.n;
  const int blk = pos0 / kKvBlock + (blockIdx.x - b * blocks_per_seq);
  const int t0 = max(pos0, blk * kKvBlock), t1 = min(s.len, (blk + 1) * kKvBlock);  // positions to read
  if (t0 >= t1) return;
  const int phys = rows.table[(long long)b * rows.W + blk];
  const bool bad = phys < 0 || phys >= n_blocks;
  if (bad && lane == 0) dev_report(ctl, DEV_ERR_BAD_BATCH, 4);
  const uint8_t* tile = tiles + ((long long)(bad ? 0 : phys) * Hkv + h) * G::TILE;
  const long long ldo = (long long)Hkv * HD;
  const long long out0 = ((long long)s.row0 - pos0) * ldo + (long long)h * HD;  // of position 0
  // NT tiles at a time, every load of theirs first
  constexpr int NT = G::BITS == 4 ? 2 : 1;
#pragma unroll 1
  for (int base0 = t0 & ~15; base0 < t1; base0 += 16 * NT) {
    unsigned int uv[NT][G::VB], uk[NT][2][G::KB / 4];
    unsigned int sv[NT][4], sk[NT][2];  // scales of this lane's four values and two keys (NG of 16 bits)
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int slot = (base0 + 16 * n) % kKvBlock, i0 = slot % kKvRec;  // (past t1: still in the tile's bytes)
      const uint8_t* rec = tile + slot / kKvRec * G::REC;
#pragma unroll
      for (int p = 0; p < G::VB / 4; ++p) {
        const uint4 x = *reinterpret_cast<const uint4*>(rec + G::VCODES + i0 * G::ROWB + p * 512 + lane * 16);
        uv[n][4 * p] = x.x, uv[n][4 * p + 1] = x.y, uv[n][4 * p + 2] = x.z, uv[n][4 * p + 3] = x.w;
      }
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
#pragma unroll
        for (int p = 0; p < G::KB / G::KP; ++p) {
          const uint8_t* at = rec + i0 * G::ROWB + p * 64 * G::KP + (r + 8 * hf) * 4 * G::KP + c * G::KP;
          if (G::KP == 16) {
            const uint4 x = *reinterpret_cast<const uint4*>(at);
            uk[n][hf][4 * p] = x.x, uk[n][hf][4 * p + 1] = x.y, uk[n][hf][4 * p + 2] = x.z, uk[n][hf][4 * p + 3] = x.w;
          } else {
            const uint2 x = *reinterpret_cast<const uint2*>(at);
            uk[n][hf][0] = x.x, uk[n][hf][1] = x.y;
          }
        }
      auto scales = [&](int off, int i) -> unsigned int {
        const uint8_t* at = rec + off + (i0 + i) * 2 * G::NG;
        return G::NG == 2 ? *reinterpret_cast<const unsigned int*>(at)
                          : *reinterpret_cast<const unsigned short*>(at);
      };
#pragma unroll
      for (int sl = 0; sl < 4; ++sl) sv[n][sl] = scales(G::VSCALE, 2 * c + (sl & 1) + 8 * (sl >> 1));
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) sk[n][hf] = scales(G::KSCALE, r + 8 * hf);
    }
    auto scale = [&](unsigned int u, int g) {
      return bad ? __uint_as_float(0x7fc00000u) : G::NG == 2 && g ? bf16_hi(u) : bf16_lo(u);
    };
    auto value = [&](unsigned int word, int i, float sf) {  // code i of the word
      const unsigned int u = (word >> (i * G::BITS)) & (2 * G::Z - 1);
      return sf * (__uint_as_float(0x4b000000u | u) - (8388608.f + G::Z));
    };
    auto pair = [&](unsigned int word, int i, float sf) {  // codes i and i + 1 as two bf16
      const __nv_bfloat162 p = __floats2bfloat162_rn(value(word, i, sf), value(word, i + 1, sf));
      return *reinterpret_cast<const unsigned int*>(&p);
    };
    auto octet = [&](const unsigned int* w, float sf) {
      return G::BITS == 4 ? make_uint4(pair(w[0], 0, sf), pair(w[0], 2, sf), pair(w[0], 4, sf), pair(w[0], 6, sf))
                          : make_uint4(pair(w[0], 0, sf), pair(w[0], 2, sf), pair(w[1], 0, sf), pair(w[1], 2, sf));
    };
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int base = base0 + 16 * n;
#pragma unroll
      for (int sl = 0; sl < 4; ++sl) {
        const int t = base + 2 * c + (sl & 1) + 8 * (sl >> 1);
        if (t >= t0 && t < t1) {
          __nv_bfloat16* out = v_out + out0 + t * ldo + 8 * r;
#pragma unroll
          for (int wj = 0; wj < HD / 64; ++wj)
            *reinterpret_cast<uint4*>(out + 64 * wj) =
                octet(uv[n] + (sl * G::VB + wj * G::BITS) / 4, scale(sv[n][sl], G::NG == 1 ? 0 : wj));
        }
      }
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int t = base + r + 8 * hf;
        if (t >= t0 && t < t1) {
          __nv_bfloat16* out = k_out + out0 + t * ldo;
#pragma unroll
          for (int wi = 0; wi < G::KB / 4; ++wi) {
            const float sf = scale(sk[n][hf], G::NG == 1 ? 0 : wi / 2);
            if (G::BITS == 4) {
              *reinterpret_cast<uint4*>(out + 32 * wi + 8 * c) = octet(&uk[n][hf][wi], sf);
            } else {
              *reinterpret_cast<uint2*>(out + 16 * wi + 4 * c) =
                  make_uint2(pair(uk[n][hf][wi], 0, sf), pair(uk[n][hf][wi], 2, sf));
            }
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
  if (b->n_seq < 0 || b->max_blocks < 1 || kv_max_new(b) < 0)
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
  if (rope && !(rope_base > 1.f && std::isfinite(rope_base)))
    return set_error(ST_INVALID_ARG, "kv_append: rope_base must be finite and > 1");
  if (qk_norm && !(eps > 0.f && std::isfinite(eps)))
    return set_error(ST_INVALID_ARG, "kv_append: eps must be finite and > 0");
  const int max_new = kv_max_new(batch);
  if (M == 0 || batch->n_seq == 0 || max_new == 0) return ST_OK;
  if (!qkv || !q_out) return set_error(ST_INVALID_ARG, "kv_append: null qkv or q_out");
  if (misaligned(qkv, 16) || misaligned(q_out, 16))
    return set_error(ST_INVALID_ARG, "kv_append: qkv and q_out must be 16-byte aligned");
  const long long bps = ((long long)max_new + kKvBlock - 2) / kKvBlock + 1;  // blocks that max_new tokens can touch
  if (bps * batch->n_seq > 0x7fffffffLL) return set_error(ST_UNSUPPORTED, "kv_append: n_seq x max_new too large");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const DevCtl ctl = device_ctl();
  if (!ctl.status) return set_error(ST_CUDA, "device status word unavailable");
  RopeFreq f;
  // powers of base^(-2 / hd), which is square roots of 1 / base, in extended precision (64 calls of pow would
  // take longer than the launch; a table of 8 x 8 as a smaller parameter saves the host 0.6 us and costs 5 % of the
  // kernel on prompts)
  long double ratio = rope ? 1.0L / rope_base : 0.0L, fi = 1.0L;
  for (int n = cache->head_dim / 2; n > 1; n /= 2) ratio = std::sqrt(ratio);
  for (int i = 0; i < 64; ++i, fi *= ratio) f.f[i] = (double)fi;
  const double row = (double)(H + 2 * Hkv) * cache->head_dim;
  Prof prof(PK_QK, 0, M * row * 2 + (double)M * H * cache->head_dim * 2, st);
  return kv_dispatch(cache, [&](auto g) -> int {
    using G = decltype(g);
    // the heads are shared among enough CTAs to give every SM four (with one, two, four and eight, 30 heads of 128:
    // 16 x 300 tokens 28.0 / 21.2 / 21.2 / 21.2 us, 64 x 300 53.8 / 53.8 / 52.7 / 50.1, 4 x 2048 28.4 / 23.0 / 21.5 / 21.5,
    // 16 x 2048 54.3 / 54.4 / 56.7 / 60.7), as far as the warps have turns: one for each head where a block can have a
    // token for each of the SG lane groups, else one for SG heads (16 x 6 new tokens 5.0 us, 9.0 with a quarter of
    // the CTAs)
    constexpr int SG = 512 / G::HD;
    const long long ctas = bps * batch->n_seq;
    const int hw = max_new >= SG ? H + 2 * Hkv : (H + 2 * Hkv + SG - 1) / SG;
    long long y = ctas >= 4LL * num_sms() ? 1 : (4LL * num_sms() + ctas - 1) / ctas;
    if (y > (hw + 7) / 8) y = (hw + 7) / 8;
    const KvRows r = kv_rows(batch, M);
    constexpr int SMEM = kKvBlock * G::HD * 4 + kAppendThreads / 32 * kAppendRing * 1024;
    static bool attr_set[64] = {};
    int dev = 0;
    GPTK_CUDA(cudaGetDevice(&dev));
    if (!attr_set[dev & 63]) {
      GPTK_CUDA(cudaFuncSetAttribute(kv_append_kernel<G>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM));
      attr_set[dev & 63] = true;
    }
    GPTK_CUDA(launch_pdl(kv_append_kernel<G>, dim3((unsigned)ctas, (unsigned)y), dim3(kAppendThreads), SMEM, st,
                         static_cast<const __nv_bfloat16*>(qkv), r, (int)bps, static_cast<uint8_t*>(cache->tiles),
                         static_cast<__nv_bfloat16*>(cache->bounds), (int)cache->n_blocks, H, Hkv, rope, qk_norm, eps, f,
                         static_cast<__nv_bfloat16*>(q_out), ctl));
    return ST_OK;
  });
}

GPT_API int gpt_op_kv_read(const gpt_kv_cache* cache, const gpt_kv_batch* batch, int M, void* k_out, void* v_out,
                           void* stream) {
  set_error(ST_OK, "");
  GPTK_TRY(kv_check("kv_read", cache, batch, M));
  const int max_new = kv_max_new(batch);
  if (M == 0 || batch->n_seq == 0 || max_new == 0) return ST_OK;
  if (!k_out || !v_out) return set_error(ST_INVALID_ARG, "kv_read: null k_out or v_out");
  if (misaligned(k_out, 16) || misaligned(v_out, 16))
    return set_error(ST_INVALID_ARG, "kv_read: k_out and v_out must be 16-byte aligned");
  const int Hkv = cache->n_kv_head;
  const long long bps = ((long long)max_new + kKvBlock - 2) / kKvBlock + 1;  // blocks that max_new tokens can touch
  if (bps * batch->n_seq > 0x7fffffffLL) return set_error(ST_UNSUPPORTED, "kv_read: n_seq x max_new too large");
  const int groups = (Hkv + 7) / 8, warps = (Hkv + groups - 1) / groups;  // heads spread evenly over the CTAs
  if (groups > 65535) return set_error(ST_UNSUPPORTED, "kv_read: too many kv heads");
  const DevCtl ctl = device_ctl();
  if (!ctl.status) return set_error(ST_CUDA, "device status word unavailable");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  Prof prof(PK_MISC, 0, (double)M * Hkv * cache->head_dim * (4 + cache->bits / 4.0), st);
  return kv_dispatch(cache, [&](auto g) -> int {
    using G = decltype(g);
    const KvRows r = kv_rows(batch, M);
    GPTK_CUDA(launch_pdl(kv_read_kernel<G>, dim3((unsigned)(bps * batch->n_seq), (unsigned)groups), dim3(32 * warps), 0,
                         st, r, (int)bps, static_cast<const uint8_t*>(cache->tiles), (int)cache->n_blocks, Hkv,
                         static_cast<__nv_bfloat16*>(k_out), static_cast<__nv_bfloat16*>(v_out), ctl));
    return ST_OK;
  });
}

}  // extern "C"
