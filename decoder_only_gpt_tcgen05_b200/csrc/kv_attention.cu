// Attention of a few new tokens over the quantised key/value cache.
//
//   o = softmax(q K^T / sqrt(hd) + mask) V,   K, V = scale (code - Z)
//
// Each visible cache row is read once per tile of 8 or 16 query rows and used for 4 hd flops a row:
// with one query row the arithmetic intensity is a few flops a byte and HBM bounds the kernel, as
// long as the codes can be turned into operands at the rate they arrive (46 four-bit codes a clock
// and SM).  That is what the kernel is built around:
//
//   - The codes are never converted.  An unsigned 4- or 8-bit code in the low bits of a half is the
//     fp16 subnormal code * 2^-24, which the tensor cores multiply exactly; unpacking is a mask (and
//     a shift for every other one).  Codes in bits 4..7 stand for 2^-20 and the factor 16 goes into
//     q, or into the result's row.  The zero point enters through the accumulator's initial value.
//   - mma.sync m16n8k16 rather than tcgen05: with one query row a 128-row MMA tile would be nearly
//     all padding, operands would have to be written back to shared memory in 16 bits (4x the bytes
//     that arrived), and the legacy tensor path has the rate to spare.  Cache rows are the M side
//     (S^T = K Q^T, O^T = V^T P^T), so a code fills one operand element and only the 8 query columns
//     are padded.
//   - A warp is a worker of its own: it takes an equal share of all (sequence, tile, head, 32-token
//     record) units, fetches its records with bulk copies into a private ring, keeps running maximum,
//     sum and output in registers, and never waits for another warp.  Every worker has the same
//     amount of work whatever the lengths; a (sequence, tile, head) that is cut between workers is
//     joined, in order, by kv_join_kernel, so results do not depend on timing.
//
// Numbers: scores, maxima, sums and outputs are fp32; q is scaled by a power of two into fp16, which
// is exact for a bf16 q down to 2^-28 of its row's largest; probabilities times the value scale are
// rounded to fp16 (2^-11; four times finer than bf16's 2^-9, below the output's own rounding).
#include <cfloat>
#include <cmath>
#include <string>

#include "kv.cuh"

namespace gptk {

struct AttendArgs {
  const __nv_bfloat16* q;
  const uint8_t* tiles;
  const int* sel;  // [M, Hkv, n_sel] listed blocks, or null: every visible one
  KvRows rows;
  int n_blocks, H, Hkv, G, n_sel, window;
  int E, QT;       // entries, and tiles of query rows a sequence (sparse: a token) has
  int RV;          // query rows of a tile that can be in use (scratch rows)
  int scanned;     // 1: prefix already holds the units before each entry (E large)
  float scale_log2;
  __nv_bfloat16* o;
  float* lse;
  long long* prefix;  // [E + 1] records of one head before entry e
  float* part_lse;    // [workers][2][RV]
  float* part_o;      // [workers][2][RV][hd]
  DevCtl ctl;
};

// One entry: a tile of query rows of one sequence, or, sparse, of one token.
struct KvEntry {
  int b, row0, rho0, nrows;  // query row rho of the tile: token row0 + rho / G, head h G + rho mod G
  int pos0;                  // position of token row0
  int jlo, nrec;             // first record and how many (sparse: two for each listed block)
  int nb;                    // visible blocks (sparse)
};

template <bool SPARSE>
__device__ __forceinline__ KvEntry kv_entry(const AttendArgs& p, int e, int RT, bool report) {
  KvEntry t;
  const int unit = e / p.QT;
  t.rho0 = (e - unit * p.QT) * RT;
  t.nrows = t.nrec = t.jlo = t.nb = t.pos0 = t.row0 = 0;
  t.b = unit;
  if (SPARSE && p.rows.cu) {
    int lo = 0, hi = p.rows.B;  // first sequence that ends after row `unit`
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (p.rows.cu[mid + 1] > unit) hi = mid;
      else lo = mid + 1;
    }
    t.b = lo;
    if (lo >= p.rows.B || p.rows.cu[lo] > unit) return t;  // a row of no sequence
  } else if (t.b >= p.rows.B) {
    return t;
  }
  const KvSeq s = kv_seq(p.rows, t.b);
  if (!s.ok) {
    if (report) dev_report(p.ctl, DEV_ERR_BAD_BATCH, 7);
    return t;
  }
  const int total = SPARSE ? p.G : s.n * p.G;
  if (t.rho0 >= total) return t;
  t.nrows = min(RT, total - t.rho0);
  t.row0 = SPARSE ? unit : s.row0;
  t.pos0 = SPARSE ? s.len - s.n + (unit - s.row0) : s.len - s.n;
  const int lo = t.pos0 + t.rho0 / p.G, hi = t.pos0 + (t.rho0 + t.nrows - 1) / p.G;
  if (SPARSE) {
    t.nb = lo / kKvBlock + 1;
    t.nrec = 2 * min(p.n_sel, t.nb);
  } else {
    t.jlo = p.window < 0 ? 0 : max(0, lo - p.window) / kKvRec;
    t.nrec = hi / kKvRec - t.jlo + 1;
  }
  return t;
}

// worker that owns unit f when `total` units are dealt to `workers` as [w total / workers, ...)
__device__ __forceinline__ long long worker_of(long long f, long long total, long long workers) {
  return ((f + 1) * workers - 1) / total;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], unsigned int a0, unsigned int a1, unsigned int a2,
                                        unsigned int a3, unsigned int b0, unsigned int b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// transpose of an 8 x 8 matrix of halves held as one mma fragment register
__device__ __forceinline__ unsigned int transpose8(unsigned int x) {
  unsigned int y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ unsigned int pack_h2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const unsigned int*>(&h);
}
__device__ __forceinline__ float2 unpack_h2(unsigned int u) {
  return __half22float2(*reinterpret_cast<const __half2*>(&u));
}
// 16 bytes of shared memory; HOLD keeps the read where it is written (a kernel short of registers)
template <bool HOLD>
__device__ __forceinline__ uint4 lds16(const uint8_t* p) {
  if (!HOLD) return *reinterpret_cast<const uint4*>(p);
  uint4 v;
  asm volatile("ld.volatile.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(smem_u32(p))
               : "memory");
  return v;
}
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float((unsigned int)(e + 127) << 23); }  // -126..127

constexpr int kAttendWarps = 4;
constexpr int kAttendMaxWorkers = 160 * 16;
constexpr int kScanSmem = 512;  // entries scanned by every CTA itself

// Ring depth and CTAs an SM: about 200 KB of shared memory in flight, far above the 44 KB an SM needs
// in flight to cover HBM's latency, split so that the register budget allows as many warps as fit.
template <class G, int NT>
struct AttendCfg {
  static constexpr int STAGES = G::REC > 8000 ? 2 : G::REC > 2200 ? 3 : 4;
  static constexpr int CTAS = NT > 1 ? 2 : 3;
  static constexpr int RING = STAGES * G::REC;
  static constexpr int SMEM = kAttendWarps * RING;
};

template <class G, int NT, bool SPARSE>
__global__ void __launch_bounds__(kAttendWarps * 32, AttendCfg<G, NT>::CTAS) kv_attend_kernel(AttendArgs p) {
  using C = AttendCfg<G, NT>;
  constexpr int HD = G::HD, NG = G::NG, RT = 8 * NT, MT = HD / 16, KW = G::KB / 4, VW = G::VB / 4;
  extern __shared__ __align__(128) uint8_t ring_all[];
  __shared__ uint64_t bars[kAttendWarps][C::STAGES];
  __shared__ int meta[kAttendWarps][C::STAGES];
  __shared__ long long s_pre[kScanSmem + 1];
  __shared__ long long s_warp[kAttendWarps];
  __shared__ KvEntry s_ent[kAttendWarps];
  __shared__ int abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gid = lane >> 2, c = lane & 3;
  if (lane == 0) {
    for (int i = 0; i < C::STAGES; ++i) mbar_init(&bars[warp][i], 1);
    fence_mbar_init();
  }
  if (tid == 0) abort_flag = 0;
  pdl_wait();
  pdl_trigger();

  // ---- the units before each entry
  const long long* pre = p.prefix;
  if (!p.scanned) {
    pre = s_pre;
    long long run = 0;
    for (int e0 = 0; e0 < p.E; e0 += kAttendWarps * 32) {
      const int e = e0 + tid;
      long long v = e < p.E ? kv_entry<SPARSE>(p, e, RT, blockIdx.x == 0).nrec : 0;
      const long long own = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += x;
      }
      if (lane == 31) s_warp[warp] = v;
      __syncthreads();
      long long before = run;
      for (int x = 0; x < kAttendWarps; ++x) {
        if (x < warp) before += s_warp[x];
        run += s_warp[x];
      }
      if (e < p.E) {
        s_pre[e] = before + v - own;
        if (blockIdx.x == 0) p.prefix[e] = before + v - own;
      }
      __syncthreads();
    }
    if (tid == 0) {
      s_pre[p.E] = run;
      if (blockIdx.x == 0) p.prefix[p.E] = run;
    }
  }
  __syncthreads();

  // ---- this warp's share
  const long long total = pre[p.E] * p.Hkv;
  const long long workers = min((long long)gridDim.x * kAttendWarps, total);
  const int w = warp * gridDim.x + blockIdx.x;  // neighbours on different SMs
  if (w >= workers) return;
  const long long ua = w * total / workers;
  const int units = (int)((w + 1) * total / workers - ua);
  uint8_t* ring = ring_all + warp * C::RING;

  // ---- the fetching iterator, C::STAGES units ahead of the computing one
  int fe, fh, fj;
  {
    int lo = 0, hi = p.E;  // last entry that starts at or before ua and is not empty
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pre[mid] * p.Hkv <= ua) lo = mid;
      else hi = mid;
    }
    fe = lo;
    const long long n = pre[fe + 1] - pre[fe], r = ua - pre[fe] * p.Hkv;
    fh = (int)(r / n);
    fj = (int)(r - fh * n);
  }
  int e = fe, h = fh, j = fj;  // the computing iterator
  int f_b, f_row, f_jlo, f_nrec, f_nb;  // of its entry: sequence, token row (sparse), records, blocks
  int f_phys = 0, f_kb = 0, f_next = -1;
  auto f_enter = [&](const KvEntry& t) {
    f_b = t.b, f_row = t.row0, f_jlo = t.jlo, f_nrec = t.nrec, f_nb = t.nb;
  };
  // loads the block number of unit (fe, fh, fj); `fresh`: the listed block was not loaded ahead
  auto look_up = [&](bool fresh) {
    int blk;
    if (SPARSE) {
      if ((fj & 1) && !fresh) {
        f_kb += f_kb >= 0 ? kKvRec : 0;
        return;
      }
      const int* list = p.sel + ((long long)f_row * p.Hkv + fh) * p.n_sel + (fj >> 1);
      blk = fresh ? list[0] : f_next;
      f_next = fj + 2 < f_nrec ? list[1] : -1;
      if (blk < 0 || blk >= f_nb) {
        f_kb = -1;
        return;
      }
      f_kb = blk * kKvBlock + (fj & 1) * kKvRec;
    } else {
      f_kb = (f_jlo + fj) * kKvRec;
      blk = f_kb / kKvBlock;
    }
    f_phys = p.rows.table[(long long)f_b * p.rows.W + blk];
  };
  int fetched = 0;
  auto fetch = [&](int stage) {  // the next unit into the stage, then on to the one after it
    if (fetched == units) return;
    if (lane == 0) {
      uint64_t* bar = &bars[warp][stage];
      if (f_kb < 0) {
        meta[warp][stage] = -1;
        mbar_arrive(bar);
      } else if (f_phys < 0 || f_phys >= p.n_blocks) {
        dev_report(p.ctl, DEV_ERR_BAD_BATCH, 8);
        meta[warp][stage] = -2;
        mbar_arrive(bar);
      } else {
        meta[warp][stage] = f_kb;
        mbar_expect_tx(bar, G::REC);
        bulk_load(ring + stage * G::REC,
                  p.tiles + ((long long)f_phys * p.Hkv + fh) * G::TILE + (f_kb / kKvRec & 1) * G::REC, G::REC, bar);
      }
    }
    if (++fetched == units) return;
    bool fresh = false;
    if (++fj == f_nrec) {
      fj = 0;
      fresh = true;
      if (++fh == p.Hkv) {
        fh = 0;
        do {
          ++fe;
        } while (pre[fe + 1] == pre[fe]);
        f_enter(kv_entry<SPARSE>(p, fe, RT, false));
      }
    }
    look_up(fresh);
  };
  {
    const KvEntry t = kv_entry<SPARSE>(p, fe, RT, false);
    if (lane == 0) s_ent[warp] = t;
    __syncwarp();
    f_enter(t);
  }
  look_up(true);
  for (int i = 0; i < C::STAGES; ++i) fetch(i);
  __syncwarp();

  // ---- state of one (entry, head)
  const int window = SPARSE ? -1 : p.window;
  unsigned int qb[NT][MT][2];
  float csum[NT][NG][2], qmul[NT][2];  // accumulator start (-Z sum q), and q's scale times log2(e) / sqrt(hd)
  int pcol[NT][2];
  float acc[NT][MT][4], m[NT][2], l[NT][2], vref = 0.f;  // vref: power of two, the values' unit
  int j_first, p_lo, p_hi;  // positions of the tile's first and last query row
  auto begin = [&]() {
    const KvEntry t = s_ent[warp];
    j_first = j;
    p_lo = t.pos0 + t.rho0 / p.G;
    p_hi = t.pos0 + (t.rho0 + t.nrows - 1) / p.G;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int n = nt * 8 + gid, rho = t.rho0 + n;
      const bool live = n < t.nrows;
      float x[HD / 4];
      unsigned int top = 0;
      const __nv_bfloat16* src =
          p.q + ((long long)(t.row0 + rho / p.G) * p.H + (long long)h * p.G + rho % p.G) * HD;
#pragma unroll
      for (int wi = 0; wi < KW; ++wi) {
        unsigned int u[4] = {0, 0, 0, 0};
        if (live) {
          if (G::BITS == 4) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(src + 32 * wi + 8 * c));
            u[0] = v.x, u[1] = v.y, u[2] = v.z, u[3] = v.w;
          } else {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(src + 16 * wi + 4 * c));
            u[0] = v.x, u[1] = v.y;
          }
        }
        constexpr int PER = 32 / G::BITS;  // dims of a word
#pragma unroll
        for (int y = 0; y < PER; ++y) {
          x[wi * PER + y] = y & 1 ? bf16_hi(u[y >> 1]) : bf16_lo(u[y >> 1]);
          top = max(top, __float_as_uint(x[wi * PER + y]) & 0x7fffffffu);
        }
      }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // the row times 2^(14 - ex) has its largest in [2^14, 2^15)
      const int ex = top == 0 ? 0 : max(-126, min((int)(top >> 23) - 127, 116));
      const int s1 = (14 - ex) / 2;
      const float f1 = exp2i(s1), f2 = exp2i(14 - ex - s1);
      const bool odd = (top >> 23) >= 127 + 117;  // beyond fp32's products, an infinity or a NaN
      float sum[NG];
#pragma unroll
      for (int g = 0; g < NG; ++g) sum[g] = 0.f;
#pragma unroll
      for (int wi = 0; wi < KW; ++wi) {
        const int g = NG == 1 ? 0 : wi / 2;
        if (G::BITS == 4) {
          float y[8];
#pragma unroll
          for (int z = 0; z < 8; ++z) y[z] = x[wi * 8 + z] * f1 * f2;
#pragma unroll
          for (int z = 0; z < 2; ++z) {  // nibbles (0, 4), (1, 5) and (2, 6), (3, 7)
            qb[nt][2 * wi + z][0] = pack_h2(y[2 * z], y[2 * z + 4]);
            qb[nt][2 * wi + z][1] = pack_h2(y[2 * z + 1] * 0.0625f, y[2 * z + 5] * 0.0625f);
            const float2 a = unpack_h2(qb[nt][2 * wi + z][0]), b = unpack_h2(qb[nt][2 * wi + z][1]);
            sum[g] += (a.x + a.y) + 16.f * (b.x + b.y);
          }
        } else {
          float y[4];
#pragma unroll
          for (int z = 0; z < 4; ++z) y[z] = x[wi * 4 + z] * f1 * f2;
          qb[nt][wi][0] = pack_h2(y[0], y[2]);
          qb[nt][wi][1] = pack_h2(y[1], y[3]);
          const float2 a = unpack_h2(qb[nt][wi][0]), b = unpack_h2(qb[nt][wi][1]);
          sum[g] += (a.x + a.y) + (b.x + b.y);
        }
      }
      const float mul = odd ? __uint_as_float(0x7fc00000u) : p.scale_log2 * exp2i(ex + 10);
      const int pos = live ? t.pos0 + rho / p.G : -1;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int from = (2 * c + i) * 4;
        qmul[nt][i] = __shfl_sync(0xffffffffu, mul, from);
        pcol[nt][i] = __shfl_sync(0xffffffffu, pos, from);
      }
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 1);
        sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 2);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          csum[nt][g][i] = __shfl_sync(0xffffffffu, sum[g], (2 * c + i) * 4) * (-G::Z * 5.9604644775390625e-8f);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) m[nt][i] = -INFINITY, l[nt][i] = 0.f;
#pragma unroll
      for (int x2 = 0; x2 < MT; ++x2)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[nt][x2][i] = 0.f;
    }
    vref = 0.f;
  };

  // ---- end of one (entry, head) in this worker: the output, or this worker's part of it
  auto finish = [&]() {
    const KvEntry t = s_ent[warp];
    const bool whole = j_first == 0 && j == t.nrec - 1;
    const int slot = j_first == 0 ? 1 : 0;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float sum = l[nt][i];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const int n = nt * 8 + 2 * c + i, rho = t.rho0 + n;
        if (n >= t.nrows) continue;
        // acc is in units of 2^-24 vref / 64; the rows of bits 4..7 in 16 times that
        const float f = sum == 0.f ? 0.f : 262144.f * vref / sum;
        const float lse2 = sum == 0.f ? -INFINITY : m[nt][i] + log2f(sum);
        const long long qrow = (long long)(t.row0 + rho / p.G) * p.H + (long long)h * p.G + rho % p.G;
        const long long prow = (long long)(w * 2 + slot) * p.RV + n;
#pragma unroll
        for (int wj = 0; wj < HD / 64; ++wj) {
          float v[8];
          if (G::BITS == 4) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              v[4 * x] = acc[nt][4 * wj + 2 * x][i] * f;
              v[4 * x + 2] = acc[nt][4 * wj + 2 * x][2 + i] * f;
              v[4 * x + 1] = acc[nt][4 * wj + 2 * x + 1][i] * (f * 0.0625f);
              v[4 * x + 3] = acc[nt][4 * wj + 2 * x + 1][2 + i] * (f * 0.0625f);
            }
          } else {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              v[2 * x] = acc[nt][4 * wj + x][i] * f;
              v[2 * x + 1] = acc[nt][4 * wj + x][2 + i] * f;
            }
          }
          if (whole) {
            uint4 u;
            unsigned int* uu = &u.x;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const __nv_bfloat162 b2 = __floats2bfloat162_rn(v[2 * x], v[2 * x + 1]);
              uu[x] = *reinterpret_cast<const unsigned int*>(&b2);
            }
            *reinterpret_cast<uint4*>(p.o + qrow * HD + 64 * wj + 8 * gid) = u;
          } else {
            float4* d = reinterpret_cast<float4*>(p.part_o + prow * HD + 64 * wj + 8 * gid);
            d[0] = make_float4(v[0], v[1], v[2], v[3]);
            d[1] = make_float4(v[4], v[5], v[6], v[7]);
          }
        }
        if (gid == 0) {
          if (!whole) p.part_lse[prow] = lse2;
          else if (p.lse) p.lse[qrow] = lse2 * 0.6931471805599453f;
        }
      }
    }
  };

  begin();
  int stage = 0, parity = 0;
  for (int u = 0; u < units; ++u) {
    if (!mbar_wait(&bars[warp][stage], parity, p.ctl, &abort_flag, 20)) {
      // give up: the copies still in flight land in this CTA's shared memory, so wait for them too
      for (int i = 1; i < C::STAGES; ++i) {
        const int st = (stage + i) % C::STAGES;
        if (u + i < fetched) mbar_wait(&bars[warp][st], st > stage ? parity : parity ^ 1, p.ctl, &abort_flag, 21);
      }
      return;
    }
    const int kb = meta[warp][stage];
    if (kb >= 0) {
      const uint8_t* rec = ring + stage * G::REC;
      const bool edge = kb + kKvRec - 1 > p_lo || (window >= 0 && kb < p_hi - window);
      // scores, S^T[key][query]
      float s[2][NT][4];
      float vs[2][2][NG];  // value scales of the keys of this lane's rows
#pragma unroll
      for (int tl = 0; tl < 2; ++tl) {
        unsigned int k0[KW], k1[KW];
#pragma unroll
        for (int x = 0; x < G::KB / G::KP; ++x) {
          const uint8_t* at = rec + tl * 16 * G::ROWB + x * 64 * G::KP + gid * 4 * G::KP + c * G::KP;
          if (G::KP == 16) {
            const uint4 a = lds16<NT == 2 && G::BITS == 8>(at), b = lds16<NT == 2 && G::BITS == 8>(at + 32 * G::KP);
            k0[4 * x] = a.x, k0[4 * x + 1] = a.y, k0[4 * x + 2] = a.z, k0[4 * x + 3] = a.w;
            k1[4 * x] = b.x, k1[4 * x + 1] = b.y, k1[4 * x + 2] = b.z, k1[4 * x + 3] = b.w;
          } else {
            const uint2 a = *reinterpret_cast<const uint2*>(at);
            const uint2 b = *reinterpret_cast<const uint2*>(at + 32 * G::KP);
            k0[0] = a.x, k0[1] = a.y, k1[0] = b.x, k1[1] = b.y;
          }
        }
        float sc[NG][NT][4];
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            sc[g][nt][0] = sc[g][nt][2] = csum[nt][g][0];
            sc[g][nt][1] = sc[g][nt][3] = csum[nt][g][1];
          }
#pragma unroll
        for (int wi = 0; wi < KW; ++wi) {
          const int g = NG == 1 ? 0 : wi / 2;
          if (G::BITS == 4) {
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              const unsigned int a = k0[wi] >> (8 * z), b = k1[wi] >> (8 * z);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma_f16(sc[g][nt], a & 0x000f000fu, b & 0x000f000fu, a & 0x00f000f0u, b & 0x00f000f0u,
                        qb[nt][2 * wi + z][0], qb[nt][2 * wi + z][1]);
            }
          } else {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_f16(sc[g][nt], k0[wi] & 0x00ff00ffu, k1[wi] & 0x00ff00ffu, (k0[wi] >> 8) & 0x00ff00ffu,
                      (k1[wi] >> 8) & 0x00ff00ffu, qb[nt][wi][0], qb[nt][wi][1]);
          }
        }
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const int i = tl * 16 + gid + 8 * hf;
          float ks[NG];
          if (NG == 2) {
            const unsigned int a = *reinterpret_cast<const unsigned int*>(rec + G::KSCALE + i * 4);
            const unsigned int b = *reinterpret_cast<const unsigned int*>(rec + G::VSCALE + i * 4);
            ks[0] = bf16_lo(a), ks[NG - 1] = bf16_hi(a);
            vs[tl][hf][0] = bf16_lo(b), vs[tl][hf][NG - 1] = bf16_hi(b);
          } else {
            ks[0] = bf16_bits(*reinterpret_cast<const unsigned short*>(rec + G::KSCALE + i * 2));
            vs[tl][hf][0] = bf16_bits(*reinterpret_cast<const unsigned short*>(rec + G::VSCALE + i * 2));
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              float x = sc[0][nt][2 * hf + q] * ks[0];
              if (NG == 2) x = fmaf(sc[NG - 1][nt][2 * hf + q], ks[NG - 1], x);
              s[tl][nt][2 * hf + q] = x * qmul[nt][q];
            }
        }
      }
      if (edge) {  // masked pairs get -inf; a key that no row of the tile sees also loses its value scale
#pragma unroll
        for (int tl = 0; tl < 2; ++tl)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const int key = kb + tl * 16 + gid + 8 * hf;
            if (key > p_hi || (window >= 0 && key < p_lo - window))
#pragma unroll
              for (int g = 0; g < NG; ++g) vs[tl][hf][g] = 0.f;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int q = 0; q < 2; ++q)
                if (key > pcol[nt][q] || (window >= 0 && key < pcol[nt][q] - window))
                  s[tl][nt][2 * hf + q] = -INFINITY;
          }
      }
      // The running maximum may lag by 8 (a factor 256 in p), and the values' unit is a power of two
      // at or above every scale seen: both move seldom, so the usual record costs one vote here.
      bool move = false;
#pragma unroll
      for (int tl = 0; tl < 2; ++tl)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int q = 0; q < 2; ++q) move |= s[tl][nt][2 * hf + q] > m[nt][q] + 8.f;
#pragma unroll
          for (int g = 0; g < NG; ++g) move |= vs[tl][hf][g] > vref;
        }
      if (__any_sync(0xffffffffu, move)) {
        float vm = 0.f;
#pragma unroll
        for (int tl = 0; tl < 2; ++tl)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf)
#pragma unroll
            for (int g = 0; g < NG; ++g) vm = fmaxf(vm, vs[tl][hf][g]);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) vm = fmaxf(vm, __shfl_xor_sync(0xffffffffu, vm, o));
        float fv = 1.f;
        if (vm > vref) {
          const int ex = min((int)(__float_as_uint(vm) >> 23) - 126, 126);
          const float nv = exp2i(max(ex, -125));
          fv = vref / nv;
          vref = nv;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float f[2];
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            float mx = m[nt][q];
#pragma unroll
            for (int tl = 0; tl < 2; ++tl) mx = fmaxf(mx, fmaxf(s[tl][nt][q], s[tl][nt][2 + q]));
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            f[q] = m[nt][q] == mx ? 1.f : ex2_approx(m[nt][q] - mx);
            m[nt][q] = mx;
            l[nt][q] *= f[q];
            f[q] *= fv;
          }
#pragma unroll
          for (int x = 0; x < MT; ++x)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[nt][x][i] *= f[i & 1];
        }
      }
      // probabilities, and times the value scale as the fp16 operand P^T[key][query]
      const float vinv = vref > 0.f ? 64.f / vref : 0.f;
      unsigned int pb[2][NG][NT][2];
#pragma unroll
      for (int tl = 0; tl < 2; ++tl)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float pr[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const float ref = m[nt][q] == -INFINITY ? 0.f : m[nt][q];
              pr[q] = ex2_approx(s[tl][nt][2 * hf + q] - ref);
              l[nt][q] += pr[q];
            }
#pragma unroll
            for (int g = 0; g < NG; ++g) {
              const float sv = vs[tl][hf][g] * vinv;
              float w0 = pr[0] * sv, w1 = pr[1] * sv;
              if (edge) {
                if (s[tl][nt][2 * hf] == -INFINITY) w0 = 0.f;
                if (s[tl][nt][2 * hf + 1] == -INFINITY) w1 = 0.f;
              }
              pb[tl][g][nt][hf] = transpose8(pack_h2(w0, w1));
            }
          }
      // O^T[dim][query] of this record, started at the zero point's share
      float corr[NG][NT][4];
      constexpr unsigned int NZ = 0x80008000u | G::Z | (G::Z << 16);
#pragma unroll
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int i = 0; i < 4; ++i) corr[g][nt][i] = 0.f;
#pragma unroll
          for (int tl = 0; tl < 2; ++tl) mma_f16(corr[g][nt], NZ, NZ, NZ, NZ, pb[tl][g][nt][0], pb[tl][g][nt][1]);
        }
      constexpr bool HALVES = NT == 2 && VW == 4;  // 8-byte reads, half of the words live (registers)
      unsigned int uv[2][G::VB];
      if (!HALVES) {
#pragma unroll
        for (int tl = 0; tl < 2; ++tl)
#pragma unroll
          for (int x = 0; x < G::VB / 4; ++x) {
            const uint4 a = *reinterpret_cast<const uint4*>(rec + G::VCODES + tl * 16 * G::ROWB + x * 512 + lane * 16);
            uv[tl][4 * x] = a.x, uv[tl][4 * x + 1] = a.y, uv[tl][4 * x + 2] = a.z, uv[tl][4 * x + 3] = a.w;
          }
      }
#pragma unroll
      for (int wj = 0; wj < VW; ++wj) {
        const int g = NG == 1 ? 0 : wj;
        if (HALVES && wj % 2 == 0) {
#pragma unroll
          for (int tl = 0; tl < 2; ++tl)
#pragma unroll
            for (int x = 0; x < 4; ++x)
              asm volatile("ld.volatile.shared.v2.u32 {%0, %1}, [%2];"
                           : "=r"(uv[tl][4 * x + wj]), "=r"(uv[tl][4 * x + (wj | 1)])
                           : "r"(smem_u32(rec + G::VCODES + tl * 16 * G::ROWB + x * 512 + lane * 16 + wj * 4))
                           : "memory");
        }
#pragma unroll
        for (int part = 0; part < 2; ++part) {  // low and high halves of the word: 4 or 2 dims each
          unsigned int x01[2], x23[2];
#pragma unroll
          for (int tl = 0; tl < 2; ++tl) {
            const unsigned int sel = part ? 0x7632u : 0x5410u;
            x01[tl] = __byte_perm(uv[tl][wj], uv[tl][VW + wj], sel);
            x23[tl] = __byte_perm(uv[tl][2 * VW + wj], uv[tl][3 * VW + wj], sel);
          }
#pragma unroll
          for (int z = 0; z < (G::BITS == 4 ? 2 : 1); ++z) {
            const unsigned int mask = G::BITS == 8 ? 0x00ff00ffu : z ? 0x00f000f0u : 0x000f000fu;
            const int x = G::BITS == 4 ? 4 * wj + 2 * part + z : 2 * wj + part;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float d[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) d[i] = z ? corr[g][nt][i] * 16.f : corr[g][nt][i];
#pragma unroll
              for (int tl = 0; tl < 2; ++tl)
                mma_f16(d, x01[tl] & mask, (x01[tl] >> 8) & mask, x23[tl] & mask, (x23[tl] >> 8) & mask,
                        pb[tl][g][nt][0], pb[tl][g][nt][1]);
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[nt][x][i] += d[i];
            }
          }
        }
      }
    } else if (kb == -2) {  // a block number out of range: the rows become NaN
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int q = 0; q < 2; ++q) l[nt][q] = __uint_as_float(0x7fc00000u);
    }
    __syncwarp();
    fetch(stage);
    __syncwarp();
    if (++stage == C::STAGES) stage = 0, parity ^= 1;
    const bool last = j == s_ent[warp].nrec - 1;
    if (last || u == units - 1) finish();
    ++j;
    if (last && u + 1 < units) {
      j = 0;
      if (++h == p.Hkv) {
        h = 0;
        do {
          ++e;
        } while (pre[e + 1] == pre[e]);
        __syncwarp();
        const KvEntry t = kv_entry<SPARSE>(p, e, RT, false);
        if (lane == 0) s_ent[warp] = t;
        __syncwarp();
      }
      begin();
    }
  }
}

// Units before each entry when there are more entries than a CTA scans by itself: one CTA.
template <bool SPARSE>
__global__ void __launch_bounds__(256) kv_scan_kernel(AttendArgs p, int RT) {
  __shared__ long long s_warp[8];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  long long run = 0;
  for (int e0 = 0; e0 < p.E; e0 += 256) {
    const int e = e0 + tid;
    long long v = e < p.E ? kv_entry<SPARSE>(p, e, RT, true).nrec : 0;
    const long long own = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += x;
    }
    if (lane == 31) s_warp[warp] = v;
    __syncthreads();
    long long before = run;
    for (int x = 0; x < 8; ++x) {
      if (x < warp) before += s_warp[x];
      run += s_warp[x];
    }
    if (e < p.E) p.prefix[e] = before + v - own;
    __syncthreads();
  }
  if (tid == 0) p.prefix[p.E] = run;
}

// Joins the parts of a query row that was cut between workers (one CTA a row), in the workers' order,
// and writes the rows that see no key: o = sum_i 2^(lse_i - max) o_i / sum_i 2^(lse_i - max).
constexpr int kJoinThreads = 256;
template <int HD, bool SPARSE>
__global__ void __launch_bounds__(kJoinThreads) kv_join_kernel(AttendArgs p, int RT, int max_workers) {
  constexpr int V = HD / 32;  // dims of a lane
  __shared__ float s_red[8];
  __shared__ float s_o[8][HD];
  pdl_wait();
  pdl_trigger();
  if (SPARSE && blockIdx.x == 0) kv_report_bad(p.rows, p.ctl, 9);
  const int n = blockIdx.x % p.RV;
  const long long seg = blockIdx.x / p.RV;
  const int e = (int)(seg / p.Hkv), h = (int)(seg - (long long)e * p.Hkv);
  const long long first = p.prefix[e], nrec = p.prefix[e + 1] - first, total = p.prefix[p.E] * p.Hkv;
  const long long workers = min((long long)max_workers, total);
  long long w0 = 0, w1 = -1;
  if (nrec > 0) {
    const long long f0 = first * p.Hkv + h * nrec;
    w0 = worker_of(f0, total, workers);
    w1 = worker_of(f0 + nrec - 1, total, workers);
    if (w0 == w1) return;  // one worker had all of it
  }
  const KvEntry t = kv_entry<SPARSE>(p, e, RT, false);
  if (n >= t.nrows) return;
  const int rho = t.rho0 + n;
  const long long qrow = (long long)(t.row0 + rho / p.G) * p.H + (long long)h * p.G + rho % p.G;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // the first worker's part is its last (slot 1), the others' their first (slot 0)
  auto part = [&](long long w) { return (w * 2 + (w == w0 ? 1 : 0)) * p.RV + n; };
  float mx = -INFINITY;
  for (long long w = w0 + tid; w <= w1; w += kJoinThreads) mx = fmaxf(mx, p.part_lse[part(w)]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  if (lane == 0) s_red[warp] = mx;
  __syncthreads();
#pragma unroll
  for (int x = 0; x < 8; ++x) mx = fmaxf(mx, s_red[x]);
  const float ref = mx == -INFINITY ? 0.f : mx;
  float acc[V], sum = 0.f;
#pragma unroll
  for (int x = 0; x < V; ++x) acc[x] = 0.f;
#pragma unroll 4
  for (long long w = w0 + warp; w <= w1; w += 8) {
    const long long r = part(w);
    const float g = ex2_approx(p.part_lse[r] - ref);
    const float* src = p.part_o + r * HD + lane * V;
    sum += g;
    if (V == 4) {
      const float4 v = *reinterpret_cast<const float4*>(src);
      acc[0] += g * v.x, acc[1] += g * v.y, acc[V - 2] += g * v.z, acc[V - 1] += g * v.w;
    } else {
      const float2 v = *reinterpret_cast<const float2*>(src);
      acc[0] += g * v.x, acc[1] += g * v.y;
    }
  }
#pragma unroll
  for (int x = 0; x < V; ++x) s_o[warp][lane * V + x] = acc[x];
  __syncthreads();
  if (lane == 0) s_red[warp] = sum;
  __syncthreads();
  if (tid < HD) {
    float total_sum = 0.f, v = 0.f;
#pragma unroll
    for (int x = 0; x < 8; ++x) total_sum += s_red[x], v += s_o[x][tid];
    p.o[qrow * HD + tid] = __float2bfloat16_rn(total_sum == 0.f ? 0.f : v / total_sum);
    if (tid == 0 && p.lse) p.lse[qrow] = total_sum == 0.f ? -INFINITY : (ref + log2f(total_sum)) * 0.6931471805599453f;
  }
}

// ------------------------------------------------------------------ host

struct AttendPlan {
  int NT, RT, QT, RV;
  long long E;
  size_t lse_off, o_off, total;
};

static int attend_plan(const char* what, const gpt_kv_cache* c, const gpt_kv_batch* b, int M, int H, int sparse,
                       AttendPlan* out) {
  const std::string w(what);
  if (H < 1 || H % c->n_kv_head) return set_error(ST_INVALID_ARG, w + ": H must be a multiple of n_kv_head");
  const long long G = H / c->n_kv_head;
  const long long max_new = b->cu_new ? b->max_new : 1;
  const long long rows = sparse ? G : max_new * G;  // query rows of a sequence (sparse: of a token) and kv head
  AttendPlan p;
  p.NT = rows <= 8 ? 1 : 2;
  p.RT = 8 * p.NT;
  const long long qt = rows > 0 ? (rows + p.RT - 1) / p.RT : 0;
  p.RV = (int)(rows < p.RT ? (rows > 0 ? rows : 1) : p.RT);
  p.E = (sparse ? (long long)M : (long long)b->n_seq) * qt;
  if (qt > 0x7fffffffLL || p.E * c->n_kv_head * p.RV > 0x7fffffffLL)
    return set_error(ST_UNSUPPORTED, w + ": too many query rows");
  p.QT = (int)qt;
  auto al = [](size_t x) { return (x + 255) & ~size_t(255); };
  p.lse_off = al((size_t)(p.E + 1) * 8);
  p.o_off = p.lse_off + al((size_t)kAttendMaxWorkers * 2 * p.RV * 4);
  p.total = p.o_off + (size_t)kAttendMaxWorkers * 2 * p.RV * c->head_dim * 4;
  *out = p;
  return ST_OK;
}

template <class G, int NT, bool SPARSE>
static int launch_attend(const AttendArgs& a, const AttendPlan& pl, double bytes, double flops, cudaStream_t st) {
  using C = AttendCfg<G, NT>;
  auto kern = kv_attend_kernel<G, NT, SPARSE>;
  static bool attr_set[64] = {};
  int dev = 0;
  GPTK_CUDA(cudaGetDevice(&dev));
  if (!attr_set[dev & 63]) {
    GPTK_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM));
    attr_set[dev & 63] = true;
  }
  int grid = num_sms() * C::CTAS;
  if (grid > kAttendMaxWorkers / kAttendWarps) grid = kAttendMaxWorkers / kAttendWarps;
  if (a.scanned) {
    Prof prof(PK_ATTN_FWD, 0, 0, st);
    GPTK_CUDA(launch_pdl(kv_scan_kernel<SPARSE>, dim3(1), dim3(256), 0, st, a, pl.RT));
  }
  {
    Prof prof(PK_ATTN_FWD, flops, bytes, st);
    GPTK_CUDA(launch_pdl(kern, dim3(grid), dim3(kAttendWarps * 32), C::SMEM, st, a));
  }
  Prof prof(PK_ATTN_FWD, 0, 0, st);
  GPTK_CUDA(launch_pdl(kv_join_kernel<G::HD, SPARSE>, dim3((unsigned)(pl.E * a.Hkv * pl.RV)), dim3(kJoinThreads), 0, st,
                       a, pl.RT, grid * kAttendWarps));
  return ST_OK;
}

}  // namespace gptk

using namespace gptk;

extern "C" {

GPT_API int gpt_op_attention_kv_scratch_size(const gpt_kv_cache* cache, const gpt_kv_batch* batch, int M, int H,
                                             int n_sel, size_t* bytes) {
  set_error(ST_OK, "");
  GPTK_TRY(kv_check("attention_kv", cache, batch, M));
  if (!bytes) return set_error(ST_INVALID_ARG, "attention_kv: null output");
  if (n_sel < 0) return set_error(ST_INVALID_ARG, "attention_kv: n_sel must be >= 0");
  AttendPlan pl;
  GPTK_TRY(attend_plan("attention_kv", cache, batch, M, H, n_sel > 0, &pl));
  *bytes = pl.total;
  return ST_OK;
}

GPT_API int gpt_op_attention_kv(const gpt_kv_cache* cache, const gpt_kv_batch* batch, const void* q, int M, int H,
                                int window, const int32_t* sel, int n_sel, void* o, float* lse, void* scratch,
                                size_t scratch_bytes, void* stream) {
  set_error(ST_OK, "");
  GPTK_TRY(kv_check("attention_kv", cache, batch, M));
  if (window < -1) return set_error(ST_INVALID_ARG, "attention_kv: window must be >= 0, or -1 for none");
  if (n_sel < 0 || (n_sel > 0) != (sel != nullptr))
    return set_error(ST_INVALID_ARG, "attention_kv: sel and n_sel go together");
  if (n_sel > 0 && window >= 0) return set_error(ST_UNSUPPORTED, "attention_kv: listed blocks take no window");
  if (n_sel > (1 << 24)) return set_error(ST_UNSUPPORTED, "attention_kv: n_sel above 2^24");
  AttendPlan pl;
  GPTK_TRY(attend_plan("attention_kv", cache, batch, M, H, n_sel > 0, &pl));
  if (pl.E == 0 || batch->n_seq == 0 || M == 0) return ST_OK;
  if (!q || !o || !scratch) return set_error(ST_INVALID_ARG, "attention_kv: null q, o or scratch");
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(o)) & 15)
    return set_error(ST_INVALID_ARG, "attention_kv: q and o must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(sel) | reinterpret_cast<uintptr_t>(lse)) & 3)
    return set_error(ST_INVALID_ARG, "attention_kv: sel and lse must be 4-byte aligned");
  if (reinterpret_cast<uintptr_t>(scratch) & 255)
    return set_error(ST_INVALID_ARG, "attention_kv: scratch must be 256-byte aligned");
  if (scratch_bytes < pl.total)
    return set_error(ST_WORKSPACE_TOO_SMALL, "attention_kv: scratch has " + std::to_string(scratch_bytes) +
                                                 " bytes, needs " + std::to_string(pl.total));
  AttendArgs a = {};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.tiles = static_cast<const uint8_t*>(cache->tiles);
  a.sel = sel;
  a.rows = kv_rows(batch, M);
  if (!batch->cu_new) a.rows.max_new = 1;
  a.n_blocks = cache->n_blocks;
  a.H = H;
  a.Hkv = cache->n_kv_head;
  a.G = H / cache->n_kv_head;
  a.n_sel = n_sel;
  a.window = window;
  a.E = (int)pl.E;
  a.QT = pl.QT;
  a.RV = pl.RV;
  a.scanned = pl.E > kScanSmem;
  a.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)cache->head_dim));
  a.o = static_cast<__nv_bfloat16*>(o);
  a.lse = lse;
  char* sp = static_cast<char*>(scratch);
  a.prefix = reinterpret_cast<long long*>(sp);
  a.part_lse = reinterpret_cast<float*>(sp + pl.lse_off);
  a.part_o = reinterpret_cast<float*>(sp + pl.o_off);
  a.ctl = device_ctl();
  if (!a.ctl.status) return set_error(ST_CUDA, "device status word unavailable");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return kv_dispatch(cache, [&](auto g) -> int {
    using G = decltype(g);
    if (n_sel > 0) {
      if (pl.NT == 1) return launch_attend<G, 1, true>(a, pl, 0, 0, st);
      return launch_attend<G, 2, true>(a, pl, 0, 0, st);
    }
    if (pl.NT == 1) return launch_attend<G, 1, false>(a, pl, 0, 0, st);
    return launch_attend<G, 2, false>(a, pl, 0, 0, st);
  });
}

}  // extern "C"
