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
//   - A warp is a worker of its own: it takes an equal share of all (sequence, tile, head, step of 32
//     or 64 tokens) units, fetches them with bulk copies into a private ring, keeps running maximum,
//     sum and output in registers, and never waits for another warp.  Every worker has the same
//     amount of work whatever the lengths; a (sequence, tile, head) that is cut between workers is
//     joined, in order, by kv_join_kernel, so results do not depend on timing.
//
// Measured (20-layer model's 10 heads of 128, replayed from a graph): 32 sequences of 16k to 32k tokens in 4
// bits 178 us, 6.0 TB/s; 64 of 65 to 2048 in 8 bits 41.4 us, 4.3 TB/s, of which 28 us are bytes and the rest start,
// join and launches; one of 2047 in 4 bits 8.3 us, all of it latency.  Several new tokens: a tile of 16 query rows
// reads and unpacks the cache once, so a chunk of n tokens of a head takes n / 16 passes over its keys (16 prompts
// of 2048 tokens 1200 us, where gpt_op_attention_fwd takes 376 for the same rows without a cache).
//
// Numbers: scores, maxima, sums and outputs are fp32; q is scaled by a power of two into fp16, which
// is exact for a bf16 q down to 2^-27 of its row's largest (8 bits: 2^-31); probabilities times the value scale are
// rounded to fp16: by 2^-11 of their size at most (bf16's step would be eight times that), or, those below
// 2^-19 of the largest value scale that the row has met (in this worker's part of its keys), by 2^-30 of that
// scale.  The unit that this goes by is each row's own: one for the tile would take 1 to 5 % off tiles of 16
// rows, but a large value that a row may not see (a newer token's, or one that has left the window) would wipe out
// that row.  The tensor cores align the terms of a product of 16 by their operands' exponents, of which a subnormal's
// counts as 2^-14: what lies below 2^-15 of the largest weight (or |q|) of the 16, times one code step, is cut off.
// Products are exact for weights down to 2^-5 and q down to 2^-8 of that largest; a result is off by at most 2^-11 of a
// code step per unit of weight, which shows where a dominant key's value is near zero.
#include <cfloat>
#include <cmath>
#include <string>

#include "kv.cuh"

namespace gptk {

// x / d for 0 <= x < 2^31 as a product and a shift, exact: m = (2^s + e) / d with e < d <= 2^(s - 31), so
// that x e / d < 2^s / d.  (The starts of these kernels are chains of such divisions, 100 clocks each
// otherwise.)
struct KvDiv {
  unsigned int m;
  int s;
  __host__ explicit KvDiv(int d = 1) {
    s = 31;
    while ((1LL << (s - 31)) < d) ++s;
    m = (unsigned int)(((1ULL << s) + d - 1) / d);
  }
  __device__ __forceinline__ int operator()(int x) const { return (int)(((unsigned long long)(unsigned int)x * m) >> s); }
};

struct AttendArgs {
  const __nv_bfloat16* q;
  const uint8_t* tiles;
  const int* sel;  // [M, Hkv, n_sel] listed blocks, or null: every visible one
  KvRows rows;
  int n_blocks, H, Hkv, G, n_sel, window;
  unsigned int block_bytes;  // of all kv heads' tiles
  int E, QT;       // entries, and tiles of query rows a sequence (sparse: a token) has
  int RV;          // query rows of a tile that can be in use (scratch rows)
  KvDiv by_qt, by_g, by_rv, by_hkv;  // x / QT, G, RV, Hkv
  int max_workers;
  unsigned long long worker_m;  // 2^64 / max_workers, rounded up
  int scanned;     // 1: prefix already holds the units before each entry (E large)
  float scale_log2;
  __nv_bfloat16* o;
  float* lse;
  long long* prefix;  // [E + 1] units of one head before entry e
  int* count;         // [E + 1] entries with units before entry e
  float* part_lse;    // [workers][2][RV]
  float* part_o;      // [workers][2][RV][hd]
  DevCtl ctl;
};

// One entry: a tile of query rows of one sequence, or, sparse, of one token.
struct KvEntry {
  int b, row0, rho0, nrows;  // query row rho of the tile: token row0 + rho / G, head h G + rho mod G
  int pos0;                  // position of token row0
  int jlo, nrec;             // first unit of U keys, and how many (sparse: 64 / U for each listed block)
  int nb;                    // visible blocks (sparse)
};

// Where a worker is: the entry, the head, the first of its units that it took, and the positions of the
// tile's first and last query row.
struct KvSpan {
  int e, h, j_first, p_lo, p_hi;
};

template <bool SPARSE>
__device__ __forceinline__ KvEntry kv_entry(const AttendArgs& p, int e, int RT, int U, bool report) {
  KvEntry t;
  const int unit = p.by_qt(e);
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
  const int lo = t.pos0 + p.by_g(t.rho0), hi = t.pos0 + p.by_g(t.rho0 + t.nrows - 1);
  if (SPARSE) {
    t.nb = lo / kKvBlock + 1;
    t.nrec = kKvBlock / U * min(p.n_sel, t.nb);
  } else {
    t.jlo = p.window < 0 ? 0 : max(0, lo - p.window) / U;
    t.nrec = hi / U - t.jlo + 1;
  }
  return t;
}

// The work is dealt out by weight: a unit weighs 1, and starting an (entry, head), with its q to load and
// its output to write, kSegWeight more, so that a worker with several short sequences gets fewer units
// (2 measured best of 0 .. 4: drafts over a window 25.2 -> 22.2 us, two drafted tokens over listed blocks
// 50.2 -> 47.1, one sequence alone 9.8 -> 10).
// Weight [w total / workers, (w + 1) total / workers) is worker w's; a segment's extra weight lies before
// its first unit.
constexpr int kSegWeight = 2;
// (64-bit division takes hundreds of clocks and is needed for huge batches only)
__device__ __forceinline__ long long div_pos(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((unsigned int)a / (unsigned int)b) : a / b;
}
__device__ __forceinline__ long long worker_of(long long weight, long long total, long long workers) {
  return div_pos((weight + 1) * workers - 1, total);
}
// w total / workers for workers = min(max_workers, total): by the reciprocal, exact while
// w total max_workers < 2^64, which is far beyond any batch that fits
__device__ __forceinline__ long long share_begin(const AttendArgs& p, int w, long long total) {
  return total <= p.max_workers ? w : (long long)__umul64hi((unsigned long long)w * total, p.worker_m);
}
// The first unit at or after weight v: its entry, head and number there, and how many units of all heads lie
// before it.  pre and cnt are the units of one head, and the non-empty entries, before each entry.
struct KvPlace {
  long long unit;
  int e, h, j;
};
__device__ __forceinline__ KvPlace unit_at(const long long* pre, const int* cnt, int E, int Hkv, long long v) {
  int lo = 0, hi = E;  // last entry whose weight begins at or before v: not an empty one, unless v is the end
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if ((pre[mid] + (long long)kSegWeight * cnt[mid]) * Hkv <= v) lo = mid;
    else hi = mid;
  }
  const long long n = pre[lo + 1] - pre[lo], r = v - (pre[lo] + (long long)kSegWeight * cnt[lo]) * Hkv;
  KvPlace at;
  at.e = lo;
  at.h = n == 0 ? 0 : (int)min(div_pos(r, n + kSegWeight), (long long)Hkv);
  at.j = max(0, (int)(r - at.h * (n + kSegWeight)) - kSegWeight);
  if (n == 0) at.j = 0;
  at.unit = pre[lo] * Hkv + at.h * n + at.j;
  return at;
}

// The units before each entry, by a whole block of W warps: into pre and cnt (and gpre and gcnt, unless
// null).  Ends with a barrier.
template <bool SPARSE, int W>
__device__ __forceinline__ void kv_scan(const AttendArgs& p, int RT, int U, bool report, long long* s_warp, int* s_wcnt,
                                        long long* pre, int* cnt, long long* gpre, int* gcnt) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  long long run = 0;
  int runc = 0;
  for (int e0 = 0; e0 < p.E; e0 += W * 32) {
    const int e = e0 + tid;
    long long v = e < p.E ? kv_entry<SPARSE>(p, e, RT, U, report).nrec : 0;
    const long long own = v;
    const unsigned int full = __ballot_sync(0xffffffffu, own > 0);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += x;
    }
    if (lane == 31) s_warp[warp] = v, s_wcnt[warp] = __popc(full);
    __syncthreads();
    long long before = run;
    int beforec = runc + __popc(full & ((1u << lane) - 1));
    for (int x = 0; x < W; ++x) {
      if (x < warp) before += s_warp[x], beforec += s_wcnt[x];
      run += s_warp[x], runc += s_wcnt[x];
    }
    if (e < p.E) {
      pre[e] = before + v - own, cnt[e] = beforec;
      if (gpre) gpre[e] = before + v - own, gcnt[e] = beforec;
    }
    __syncthreads();
  }
  if (tid == 0) {
    pre[p.E] = run, cnt[p.E] = runc;
    if (gpre) gpre[p.E] = run, gcnt[p.E] = runc;
  }
  __syncthreads();
}

// d = A B + c
__device__ __forceinline__ void mma_f16(float (&d)[4], unsigned int a0, unsigned int a1, unsigned int a2,
                                        unsigned int a3, const unsigned int (&b)[2], const float (&c)[4]) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, "
      "%12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b[0]), "r"(b[1]), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}
// d += A B
__device__ __forceinline__ void mma_f16(float (&d)[4], unsigned int a0, unsigned int a1, unsigned int a2,
                                        unsigned int a3, const unsigned int (&b)[2]) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b[0]), "r"(b[1]));
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
// bytes 1 and 3, each in the low half of 16 bits
__device__ __forceinline__ unsigned int odd_bytes(unsigned int x) { return __byte_perm(x, 0, 0x4341); }
// Shared-memory reads by 32-bit address, kept where they are written: hoisted by the compiler they
// would all be live at once, and the kernel is short of registers.
__device__ __forceinline__ void lds16(uint32_t a, unsigned int* v) {
  asm volatile("ld.volatile.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void lds8(uint32_t a, unsigned int* v) {
  asm volatile("ld.volatile.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(a) : "memory");
}
__device__ __forceinline__ unsigned int lds4(uint32_t a) {
  unsigned int v;
  asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ unsigned int lds2(uint32_t a) {
  unsigned short v;
  asm volatile("ld.volatile.shared.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float((unsigned int)(e + 127) << 23); }  // -126..127

constexpr int kAttendMaxWorkers = 160 * 16;
// Entries scanned by every CTA itself; more have a launch of their own (8 bits, 2 heads: 64 sequences 18.6 us
// against 19.9 with that launch, 256 20.1 against 21.0, 500 30.6 against 30.2).
constexpr int kScanSmem = 512;

constexpr int kSmShared = 228 * 1024;  // of an SM
constexpr int kAttendStages = 2;       // units of a warp's ring

// What a CTA of W warps with tiles of RT query rows has in shared memory beside its rings.  What is the same
// for a whole (entry, head), of the computing and the fetching iterator, lives here, written by lane 0, since
// the registers are needed for the step.
template <int W, int RT>
struct __align__(128) AttendShared {
  long long pre[kScanSmem + 1];
  int cnt[kScanSmem + 1];
  uint64_t bars[W][kAttendStages];
  int meta[W][kAttendStages];  // of a stage's unit: first key; -1: none; -2 - first key: bad block
  long long scan_units[W];
  int scan_cnt[W];
  KvEntry ent[W], fent[W];
  KvSpan span[W];
  int pos[W][RT];
  long long row[W][RT];
  int abort_flag;
};

// Keys of a unit (U) and CTAs an SM.  A unit is one fetch: 64 keys, or 32 for 128-wide
// 8-bit rows, whose 64 would leave room for too few warps.  The rings hold 100 to 200 KB an SM, far above
// the 44 KB that cover HBM's latency; 12 warps an SM leave each thread the 168 registers that one query
// column tile needs (and two of 64-wide rows), 8 warps the 255 of two; 16 warps fit with small rings only.
// A CTA that does not fit runs after the others, with a full share of the work: 64 sequences of 2k to 8k
// tokens, heads of 64: 8 bits, 12 kv heads 104 us with four CTAs launched an SM, of which three fit, 96 with
// three; 4 bits, 16 query rows 46 us with three launched of four stages, of which two fit, 33 with two, 32
// with three of two stages.
template <class G, int NT>
struct AttendCfg {
  static constexpr int U = G::REC > 8000 ? 32 : 64;
  static constexpr int WARPS = 4;
  static constexpr int CTAS = NT > 1 ? (G::HD == 64 ? 3 : 2) : (G::HD == 64 && G::BITS == 4 ? 4 : 3);
  static constexpr int STAGE = U / kKvRec * G::REC;
  static constexpr int STAGES = kAttendStages;
  static constexpr int RING = STAGES * STAGE;
  static constexpr int SMEM = WARPS * RING;
  // the rings, what else a CTA holds in shared memory, and 1 KB that the system takes of each
  static_assert(CTAS * (SMEM + sizeof(AttendShared<WARPS, 8 * NT>) + 1024) <= kSmShared, "every CTA must be resident");
};

// NT tiles of 8 query columns.  A lane's part of a product's output is two neighbouring columns: QC = 1
// uses the even ones alone, for tiles of at most four query rows (a step of a model without shared kv
// heads has one), and leaves out half of the softmax's and the output's arithmetic and registers.  A
// step then takes a whole unit (TL tiles), a record with all columns, half of one with two column tiles:
// what fits the registers (8 bits at 128 dims have one scale a row, which leaves room for a record: 16
// chunks of 512 tokens over 2k to 8k 1164 us, with half of one 1232; at 64 dims it spills).  (32 sequences of 16k to 32k tokens in 4
// bits: 212 us with both columns and a record a step, 198 with one, 185 with one and 64 keys a step, when that was
// built.)
template <class G, int NT, int QC, bool SPARSE>
__global__ void __launch_bounds__(AttendCfg<G, NT>::WARPS * 32, AttendCfg<G, NT>::CTAS) kv_attend_kernel(AttendArgs p) {
  using C = AttendCfg<G, NT>;
  constexpr int HD = G::HD, NG = G::NG, RT = 4 * QC * NT, MT = HD / 16, KW = G::KB / 4, VW = G::VB / 4;
  // with one column used, a column pair's other half carries the weights of the second scale group
  constexpr int PG = QC == 1 ? 1 : NG;  // operands P a key tile
  constexpr int U = C::U;  // keys of a unit
  constexpr bool IN_KS = NG <= NT * QC;  // where the scores' constant factor goes
  constexpr int TL = NT == 2 ? (G::BITS == 8 && HD == 128 ? 2 : 1) : QC == 2 ? 2 : U / 16;  // 16-key tiles of a step
  extern __shared__ __align__(128) uint8_t ring_all[];
  __shared__ AttendShared<C::WARPS, 8 * NT> sh;
  auto &bars = sh.bars;
  auto &meta = sh.meta;
  auto &s_ent = sh.ent, &s_fent = sh.fent;
  auto &s_span = sh.span;
  auto &s_pos = sh.pos;
  auto &s_row = sh.row;
  int& abort_flag = sh.abort_flag;
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
  const int* cnt = p.count;
  if (!p.scanned) {
    pre = sh.pre, cnt = sh.cnt;
    const bool first = blockIdx.x == 0;
    kv_scan<SPARSE, C::WARPS>(p, RT, U, first, sh.scan_units, sh.scan_cnt, sh.pre, sh.cnt, first ? p.prefix : nullptr, p.count);
  } else {
    __syncthreads();
  }

  // ---- this warp's share
  const long long total = (pre[p.E] + (long long)kSegWeight * cnt[p.E]) * p.Hkv;
  const int w = warp * gridDim.x + blockIdx.x;  // neighbours on different SMs
  if (w >= total) return;  // (there are max_workers warps)
  // (the even lanes find its beginning, the odd ones its end)
  const KvPlace place = unit_at(pre, cnt, p.E, p.Hkv, share_begin(p, w + (lane & 1), total));
  const int units = (int)(__shfl_sync(0xffffffffu, place.unit, 1) - __shfl_sync(0xffffffffu, place.unit, 0));
  if (units == 0) return;

  // ---- the fetching iterator, C::STAGES units ahead of the computing one
  int fe = __shfl_sync(0xffffffffu, place.e, 0), fh = __shfl_sync(0xffffffffu, place.h, 0);
  int fj = __shfl_sync(0xffffffffu, place.j, 0);
  int j = fj;  // the computing iterator's unit; its entry and head are in sp
  KvSpan& sp = s_span[warp];
  const KvEntry& ft = s_fent[warp];
  const uint32_t bar0 = smem_u32(&bars[warp][0]), ring0 = smem_u32(ring_all) + warp * C::RING;
  int f_phys = 0, f_kb = 0, f_tab = 0, f_next = -1;
  // the block number of unit (fe, fh, fj): after the first of a head, what changes is added up
  auto look_up = [&](bool fresh) {
    if (fresh) f_tab = ft.b * p.rows.W;
    if (SPARSE) {
      constexpr int PER = kKvBlock / U;  // units of a listed block
      if (fj % PER && !fresh) {
        f_kb += f_kb >= 0 ? U : 0;
        return;
      }
      const int* list = p.sel + ((long long)ft.row0 * p.Hkv + fh) * p.n_sel + fj / PER;
      const int blk = fresh ? list[0] : f_next;
      f_next = fj + PER < ft.nrec ? list[1] : -1;
      if (blk < 0 || blk >= ft.nb) {
        f_kb = -1;
        return;
      }
      f_kb = blk * kKvBlock + fj % PER * U;
    } else {
      f_kb = fresh ? (ft.jlo + fj) * U : f_kb + U;
    }
    f_phys = p.rows.table[f_tab + f_kb / kKvBlock];
  };
  auto fetch = [&](int f) {  // this worker's unit f into its stage, then on to the one after it
    if (f >= units) return;
    const int stage = f % C::STAGES;
    if (lane == 0) {
      const uint32_t bar = bar0 + 8 * stage;
      const bool ok = (unsigned int)f_phys < (unsigned int)p.n_blocks;
      meta[warp][stage] = f_kb < 0 ? -1 : ok ? f_kb : -2 - f_kb;
      if (f_kb >= 0 && ok) {
        const uint8_t* src = p.tiles + (unsigned long long)f_phys * p.block_bytes +
                             (unsigned int)(fh * G::TILE + (U == 64 ? 0 : f_kb / kKvRec % 2 * G::REC));
        bulk_load(ring0 + stage * C::STAGE, src, C::STAGE, bar);
      } else {
        if (f_kb >= 0) dev_report(p.ctl, DEV_ERR_BAD_BATCH, 8);
        mbar_arrive(&bars[warp][stage]);
      }
    }
    if (f + 1 >= units) return;
    bool fresh = false;
    if (++fj == ft.nrec) {
      fj = 0;
      fresh = true;
      if (++fh == p.Hkv) {
        fh = 0;
        do {
          ++fe;
        } while (pre[fe + 1] == pre[fe]);
        __syncwarp();
        const KvEntry t = kv_entry<SPARSE>(p, fe, RT, U, false);
        if (lane == 0) s_fent[warp] = t;
        __syncwarp();
      }
    }
    look_up(fresh);
  };
  {
    const KvEntry t = kv_entry<SPARSE>(p, fe, RT, U, false);
    if (lane == 0) s_ent[warp] = s_fent[warp] = t, sp.e = fe, sp.h = fh;
    __syncwarp();
  }
  look_up(true);
  for (int i = 0; i < C::STAGES; ++i) fetch(i);
  __syncwarp();

  // ---- state of one (entry, head)
  const int window = SPARSE ? -1 : p.window;
  unsigned int qb[NT][MT][2];
  float csum[NT][NG][4], qmul[NT][QC];  // accumulator start (-Z sum q), and q's scale, a power of two
  // vinv: 64 / (the values' unit of the row), a power of two, at most 2^118; vinv_top: the rows' largest
  float acc[NT][MT][2 * QC], m[NT][QC], l[NT][QC], vinv[NT][QC], vinv_top;
  auto begin = [&]() {
    const KvEntry t = s_ent[warp];
    if (lane == 0) {
      sp.j_first = j;
      sp.p_lo = t.pos0 + p.by_g(t.rho0);
      sp.p_hi = t.pos0 + p.by_g(t.rho0 + t.nrows - 1);
    }
    if (lane < RT) {  // the tile's query rows: position and row of q and o (-1: none)
      const int tok = p.by_g(t.rho0 + lane), g = t.rho0 + lane - tok * p.G;
      s_pos[warp][lane] = lane < t.nrows ? t.pos0 + tok : -1;
      s_row[warp][lane] = lane < t.nrows ? (long long)(t.row0 + tok) * p.H + sp.h * p.G + g : -1;
    }
    __syncwarp();
    constexpr int PER = 32 / G::BITS;  // dims of a code word
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const long long row = QC == 1 ? (gid % 2 ? -1 : s_row[warp][gid / 2]) : s_row[warp][nt * 8 + gid];
      unsigned int xw[HD / 8];  // this lane's quarter of the row as bf16 pairs
#pragma unroll
      for (int wi = 0; wi < KW; ++wi) {
        const __nv_bfloat16* src = p.q + row * HD + 4 * PER * wi + PER * c;
        if (G::BITS == 4) {
          const uint4 v = row >= 0 ? *reinterpret_cast<const uint4*>(src) : make_uint4(0, 0, 0, 0);
          xw[4 * wi] = v.x, xw[4 * wi + 1] = v.y, xw[4 * wi + 2] = v.z, xw[4 * wi + 3] = v.w;
        } else {
          const uint2 v = row >= 0 ? *reinterpret_cast<const uint2*>(src) : make_uint2(0, 0);
          xw[2 * wi] = v.x, xw[2 * wi + 1] = v.y;
        }
      }
      unsigned int top = 0;  // largest |x| as bits
#pragma unroll
      for (int i = 0; i < HD / 8; ++i) top = max(top, max((xw[i] << 16) & 0x7fffffffu, xw[i] & 0x7fff0000u));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // the row times 2^(14 - ex) has its largest in [2^14, 2^15)
      const int ex = top == 0 ? 0 : max(-126, min((int)(top >> 23) - 127, 116));
      const int s1 = (14 - ex) / 2;
      const float f1 = exp2i(s1), f2 = exp2i(14 - ex - s1);
      const bool odd = (top >> 23) >= 127 + 117;  // beyond fp32's products, an infinity or a NaN
      auto y = [&](int i) { return (i & 1 ? bf16_hi(xw[i >> 1]) : bf16_lo(xw[i >> 1])) * f1 * f2; };
      float sum[NG];
#pragma unroll
      for (int g = 0; g < NG; ++g) sum[g] = 0.f;
#pragma unroll
      for (int k = 0; k < MT; ++k) {
        const int g = NG == 1 ? 0 : k / 4;
        unsigned int(&b)[2] = qb[nt][k];
        if (G::BITS == 4) {  // word k / 2: nibbles (0, 4), (1, 5) or (2, 6), (3, 7)
          const int at = k / 2 * 8 + k % 2 * 2;
          b[0] = pack_h2(y(at), y(at + 4));
          b[1] = pack_h2(y(at + 1) * 0.0625f, y(at + 5) * 0.0625f);
        } else {  // word k: bytes (0, 2), (1, 3)
          b[0] = pack_h2(y(4 * k), y(4 * k + 2));
          b[1] = pack_h2(y(4 * k + 1), y(4 * k + 3));
        }
        const float2 u = unpack_h2(b[0]), v = unpack_h2(b[1]);
        sum[g] += (u.x + u.y) + (G::BITS == 4 ? 16.f : 1.f) * (v.x + v.y);
      }
      const float mul = odd ? __uint_as_float(0x7fc00000u) : exp2i(ex + 10);
#pragma unroll
      for (int i = 0; i < QC; ++i) qmul[nt][i] = __shfl_sync(0xffffffffu, mul, (2 * c + i) * 4);
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 1);
        sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 2);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          csum[nt][g][i] = csum[nt][g][2 + i] =
              __shfl_sync(0xffffffffu, sum[g], (2 * c + i) * 4) * (-G::Z * 5.9604644775390625e-8f);
      }
#pragma unroll
      for (int i = 0; i < QC; ++i) m[nt][i] = -FLT_MAX, l[nt][i] = 0.f, vinv[nt][i] = vinv_top = exp2i(118);
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int k = 0; k < 2 * QC; ++k) acc[nt][i][k] = 0.f;
    }
  };

  // ---- end of one (entry, head) in this worker: the output, or this worker's part of it
  auto finish = [&]() {
    const bool whole = sp.j_first == 0 && j == s_ent[warp].nrec - 1;
    const long long part0 = ((long long)(warp * gridDim.x + blockIdx.x) * 2 + (sp.j_first == 0 ? 1 : 0)) * p.RV;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < QC; ++i) {
        float sum = l[nt][i];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const int n = QC == 1 ? c : nt * 8 + 2 * c + i;
        const long long qrow = s_row[warp][n];
        if (qrow >= 0) {
          // acc is in units of 2^-24 / vinv; the rows of bits 4..7 in 16 times that
          const float f = sum == 0.f ? 0.f : 16777216.f / sum, fi = 1.f / vinv[nt][i];
          const float lse2 = sum == 0.f ? -INFINITY : m[nt][i] + log2f(sum);
#pragma unroll
          for (int wj = 0; wj < HD / 64; ++wj) {
            float v[8];
            if (G::BITS == 4) {
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                v[4 * x] = acc[nt][4 * wj + 2 * x][i] * f * fi;
                v[4 * x + 2] = acc[nt][4 * wj + 2 * x][QC + i] * f * fi;
                v[4 * x + 1] = acc[nt][4 * wj + 2 * x + 1][i] * (f * 0.0625f) * fi;
                v[4 * x + 3] = acc[nt][4 * wj + 2 * x + 1][QC + i] * (f * 0.0625f) * fi;
              }
            } else {
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                v[2 * x] = acc[nt][4 * wj + x][i] * f * fi;
                v[2 * x + 1] = acc[nt][4 * wj + x][QC + i] * f * fi;
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
              float4* d = reinterpret_cast<float4*>(p.part_o + (part0 + n) * HD + 64 * wj + 8 * gid);
              d[0] = make_float4(v[0], v[1], v[2], v[3]);
              d[1] = make_float4(v[4], v[5], v[6], v[7]);
            }
          }
          if (gid == 0) {
            if (!whole) p.part_lse[part0 + n] = lse2;
            else if (p.lse) p.lse[qrow] = lse2 * 0.6931471805599453f;
          }
        }
        __syncwarp();
      }
    }
  };

  begin();
  for (int u = 0; u < units; ++u) {
    const int stage = u % C::STAGES;
    if (!mbar_wait(&bars[warp][stage], u / C::STAGES & 1, p.ctl, &abort_flag, 20)) {
      // give up: the copies of units u .. u + STAGES - 1 may still be in flight into this CTA's shared memory
      const uint64_t t0 = globaltimer();
      for (int i = u; i < u + C::STAGES && i < units; ++i)
        mbar_drain(&bars[warp][i % C::STAGES], i / C::STAGES & 1, p.ctl, t0);
      return;
    }
    const int kb0 = meta[warp][stage];
    const int p_hi = sp.p_hi;
    // the unit's steps (none for a unit that was not fetched)
#pragma unroll 1
    for (int st = 0; st < (kb0 < 0 ? 0 : U / (16 * TL)); ++st) {
      const int kb = kb0 + st * 16 * TL;
      if (kb > p_hi) break;
      const uint32_t rec = ring0 + stage * C::STAGE + st * TL / 2 * G::REC;
      const uint32_t tile0 = st * TL % 2;  // of the record; 0 unless a step is half of one
      const uint32_t kaddr = rec + tile0 * 16 * G::ROWB + gid * 4 * G::KP + c * G::KP;
      const uint32_t saddr = rec + G::KSCALE + tile0 * 16 * 2 * NG + gid * 2 * NG;
      const uint32_t va = rec + G::VCODES + tile0 * 16 * G::ROWB + lane * 16;
      const bool edge = kb + 16 * TL - 1 > sp.p_lo || (window >= 0 && kb < p_hi - window);
      // scores S^T[key][query] but for q's scale, and the value scales of the keys of this lane's rows.  The factor
      // log2(e) / sqrt(hd) goes into the key's scales, or, where that is less to multiply, into the score; what is
      // left is a power of two, so the largest score is the maximum to the last bit (rounded apart from it, scores
      // beyond 2^31 gave p = 2^256)
      float x[TL][NT][2 * QC];
      unsigned int vs[TL][2];
#pragma unroll
      for (int tl = 0; tl < TL; ++tl) {
        const uint32_t ka = kaddr + tl / 2 * G::REC + tl % 2 * 16 * G::ROWB;
        unsigned int k0[KW], k1[KW];
#pragma unroll
        for (int y = 0; y < G::KB / G::KP; ++y) {
          if (G::KP == 16) {
            lds16(ka + y * 64 * G::KP, &k0[4 * y]);
            lds16(ka + y * 64 * G::KP + 32 * G::KP, &k1[4 * y]);
          } else {
            lds8(ka, k0);
            lds8(ka + 32 * G::KP, k1);
          }
        }
        float sc[NG][NT][4];
#pragma unroll
        for (int wi = 0; wi < KW; ++wi) {
          const int g = NG == 1 ? 0 : wi / 2;
          const bool first = NG == 1 ? wi == 0 : wi % 2 == 0;
#pragma unroll
          for (int z = 0; z < (G::BITS == 4 ? 2 : 1); ++z) {
            const unsigned int m0 = G::BITS == 4 ? 0x000f000fu : 0x00ff00ffu, m1 = G::BITS == 4 ? 0x00f000f0u : m0;
            const unsigned int a = z ? k0[wi] >> 8 : k0[wi], b = z ? k1[wi] >> 8 : k1[wi];
            const unsigned int a2 = G::BITS == 4 ? a & m1 : odd_bytes(k0[wi]), a3 = G::BITS == 4 ? b & m1 : odd_bytes(k1[wi]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const unsigned int(&qf)[2] = qb[nt][G::BITS == 4 ? 2 * wi + z : wi];
              if (first && z == 0) mma_f16(sc[g][nt], a & m0, b & m0, a2, a3, qf, csum[nt][g]);
              else mma_f16(sc[g][nt], a & m0, b & m0, a2, a3, qf);
            }
          }
        }
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const uint32_t sa = saddr + tl / 2 * G::REC + (tl % 2 * 16 + 8 * hf) * 2 * NG;
          float ks[NG];
          if (NG == 2) {
            const unsigned int a = lds4(sa);
            ks[0] = bf16_lo(a), ks[NG - 1] = bf16_hi(a);
            vs[tl][hf] = lds4(sa + G::VSCALE - G::KSCALE);
          } else {
            ks[0] = bf16_bits(lds2(sa));
            vs[tl][hf] = lds2(sa + G::VSCALE - G::KSCALE);
          }
          if (IN_KS) {
#pragma unroll
            for (int g = 0; g < NG; ++g) ks[g] *= p.scale_log2;
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int q = 0; q < QC; ++q) {
              float v = sc[0][nt][2 * hf + q] * ks[0];
              if (NG == 2) v = fmaf(sc[NG - 1][nt][2 * hf + q], ks[NG - 1], v);
              x[tl][nt][QC * hf + q] = IN_KS ? v : v * p.scale_log2;
            }
        }
      }
      // The running maximum may lag by 8 (a factor 256 in p), and the values' unit is a power of two at or
      // above every scale that the row has seen: both move seldom, so the usual step costs one vote here.
      float xm[NT][QC], vm[NT][QC];
      auto pair = [&](int tl, int hf) { return *reinterpret_cast<const __nv_bfloat162*>(&vs[tl][hf]); };
      if (edge) {  // masked pairs get -inf, and their scales do not count
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int q = 0; q < QC; ++q) vm[nt][q] = 0.f;
#pragma unroll
        for (int tl = 0; tl < TL; ++tl)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const int key = kb + tl * 16 + gid + 8 * hf;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int q = 0; q < QC; ++q) {
                const int pos = s_pos[warp][QC == 1 ? c : nt * 8 + 2 * c + q];
                if (key > pos || (window >= 0 && key < pos - window)) x[tl][nt][QC * hf + q] = -INFINITY;
                else vm[nt][q] = fmaxf(vm[nt][q], fmaxf(bf16_lo(vs[tl][hf]), bf16_hi(vs[tl][hf])));
              }
          }
      } else {
        __nv_bfloat162 v2 = __hmax2(pair(0, 0), pair(0, 1));
#pragma unroll
        for (int tl = 1; tl < TL; ++tl) v2 = __hmax2(v2, __hmax2(pair(tl, 0), pair(tl, 1)));
        const float v = fmaxf(__low2float(v2), __high2float(v2));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int q = 0; q < QC; ++q) vm[nt][q] = v;
      }
      bool move = false;
      float vm_top = 0.f;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int q = 0; q < QC; ++q) {
          xm[nt][q] = x[0][nt][q];
#pragma unroll
          for (int tl = 0; tl < TL; ++tl) xm[nt][q] = fmaxf(fmaxf(xm[nt][q], x[tl][nt][q]), x[tl][nt][QC + q]);
          move |= fmaf(xm[nt][q], qmul[nt][q], -m[nt][q]) > 8.f;
          vm_top = fmaxf(vm_top, vm[nt][q]);
        }
      move |= vm_top * vinv_top > 64.f;
      if (__any_sync(0xffffffffu, move)) {
        vinv_top = 0.f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float f[QC];
#pragma unroll
          for (int q = 0; q < QC; ++q) {
            float mx = xm[nt][q], v = vm[nt][q];
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
              v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
            }
            mx = fmaxf(m[nt][q], mx * qmul[nt][q]);
            f[q] = m[nt][q] == mx ? 1.f : ex2_approx(m[nt][q] - mx);
            m[nt][q] = mx;
            l[nt][q] *= f[q];
            if (v * vinv[nt][q] > 64.f) {  // the unit becomes the power of two above v
              const float nv = exp2i(max(6 - ((int)(__float_as_uint(v) >> 23) - 126), -121));
              f[q] *= nv / vinv[nt][q];
              vinv[nt][q] = nv;
            }
            vinv_top = fmaxf(vinv_top, vinv[nt][q]);
          }
#pragma unroll
          for (int y = 0; y < MT; ++y)
#pragma unroll
            for (int i = 0; i < 2 * QC; ++i) acc[nt][y][i] *= f[i % QC];
        }
      }
      // probabilities, and times the value scale as the fp16 operand P^T[key][query]
      unsigned int pb[TL][PG][NT][2];
#pragma unroll
      for (int tl = 0; tl < TL; ++tl)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const float sc[2] = {bf16_lo(vs[tl][hf]), bf16_hi(vs[tl][hf])};  // (the second is 0 with one scale a row)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float pr[QC];
#pragma unroll
            for (int q = 0; q < QC; ++q) {
              pr[q] = ex2_approx(fmaf(x[tl][nt][QC * hf + q], qmul[nt][q], -m[nt][q]));
              l[nt][q] += pr[q];
            }
#pragma unroll
            for (int g = 0; g < PG; ++g) {
              float w[2] = {0.f, 0.f};  // (pr vinv is at most 2^126)
              if (QC == 1) {
#pragma unroll
                for (int k = 0; k < NG; ++k)
                  w[k] = edge && x[tl][nt][hf] == -INFINITY ? 0.f : pr[0] * vinv[nt][0] * sc[k];
              } else {
#pragma unroll
                for (int q = 0; q < QC; ++q)
                  w[q] = edge && x[tl][nt][QC * hf + q] == -INFINITY ? 0.f : pr[q] * vinv[nt][q] * sc[g];
              }
              pb[tl][g][nt][hf] = transpose8(pack_h2(w[0], w[1]));
            }
          }
        }
      // O^T[dim][query] of this step, started at the zero point's share: -Z sum of the weights, from a
      // product with a constant operand (16 times that where the codes are in bits 4..7)
      constexpr int NZ = G::BITS == 4 ? 2 : 1;
      // words of the step's values: [tile][slot (key of the lane)][word]
      constexpr bool HALVES = VW == 4;  // 8-byte reads, half of the words live (registers)
      float corr[NZ][NT][4];
      {
        unsigned int uv[TL][G::VB];
        if (!HALVES) {
#pragma unroll
          for (int tl = 0; tl < TL; ++tl)
#pragma unroll
            for (int y = 0; y < G::VB / 4; ++y) lds16(va + tl / 2 * G::REC + tl % 2 * 16 * G::ROWB + y * 512, &uv[tl][4 * y]);
        }
#pragma unroll
        for (int wj = 0; wj < VW; ++wj) {
          const int g = PG == 1 ? 0 : wj;       // operand P
          const int k = QC == 1 && NG == 2 ? wj : 0;  // its column
          if (wj == 0 || PG == 2) {
            constexpr unsigned int ZC = 0x80008000u | G::Z | (G::Z << 16);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const float zero[4] = {0.f, 0.f, 0.f, 0.f};
              mma_f16(corr[0][nt], ZC, ZC, ZC, ZC, pb[0][g][nt], zero);
#pragma unroll
              for (int tl = 1; tl < TL; ++tl) mma_f16(corr[0][nt], ZC, ZC, ZC, ZC, pb[tl][g][nt]);
              if (NZ == 2) {
#pragma unroll
                for (int i = 0; i < 4; ++i) corr[NZ - 1][nt][i] = 16.f * corr[0][nt][i];
              }
            }
          }
          if (HALVES && wj % 2 == 0) {
#pragma unroll
            for (int tl = 0; tl < TL; ++tl)
#pragma unroll
              for (int y = 0; y < 4; ++y) lds8(va + tl / 2 * G::REC + tl % 2 * 16 * G::ROWB + y * 512 + wj * 4, &uv[tl][4 * y + wj]);
          }
#pragma unroll
          for (int part = 0; part < 2; ++part) {  // low and high halves of the word: 4 or 2 dims each
            unsigned int x01[TL], x23[TL];
#pragma unroll
            for (int tl = 0; tl < TL; ++tl) {
              const unsigned int sel = part ? 0x7632u : 0x5410u;
              x01[tl] = __byte_perm(uv[tl][wj], uv[tl][VW + wj], sel);
              x23[tl] = __byte_perm(uv[tl][2 * VW + wj], uv[tl][3 * VW + wj], sel);
            }
#pragma unroll
            for (int z = 0; z < NZ; ++z) {
              const unsigned int mask = G::BITS == 8 ? 0x00ff00ffu : z ? 0x00f000f0u : 0x000f000fu;
              auto second = [&](unsigned int x) { return G::BITS == 8 ? odd_bytes(x) : (x >> 8) & mask; };
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                float d[4];
                mma_f16(d, x01[0] & mask, second(x01[0]), x23[0] & mask, second(x23[0]), pb[0][g][nt], corr[z][nt]);
#pragma unroll
                for (int tl = 1; tl < TL; ++tl)
                  mma_f16(d, x01[tl] & mask, second(x01[tl]), x23[tl] & mask, second(x23[tl]), pb[tl][g][nt]);
                float(&o)[2 * QC] = acc[nt][G::BITS == 4 ? 4 * wj + 2 * part + z : 2 * wj + part];
                if (QC == 1) {
                  o[0] += d[k], o[1] += d[2 + k];
                } else {
                  const float2 s0 = fadd2(make_float2(o[0], o[1]), make_float2(d[0], d[1]));
                  const float2 s1 = fadd2(make_float2(o[2 * QC - 2], o[2 * QC - 1]), make_float2(d[2], d[3]));
                  o[0] = s0.x, o[1] = s0.y, o[2 * QC - 2] = s1.x, o[2 * QC - 1] = s1.y;
                }
              }
            }
          }
        }
      }
    }
    if (kb0 < -1) {  // a block number out of range: the rows that see one of the unit's keys become NaN
      const int kb = -2 - kb0;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int q = 0; q < QC; ++q) {
          const int pos = s_pos[warp][QC == 1 ? c : nt * 8 + 2 * c + q];
          if (kb <= pos && (window < 0 || kb + U - 1 >= pos - window)) l[nt][q] = __uint_as_float(0x7fc00000u);
        }
    }
    __syncwarp();
    fetch(u + C::STAGES);
    __syncwarp();
    const bool last = j == s_ent[warp].nrec - 1;
    if (last || u == units - 1) finish();
    ++j;
    if (last && u + 1 < units) {
      j = 0;
      int e = sp.e, h = sp.h + 1;
      const bool turn = h == p.Hkv;
      if (turn) {
        h = 0;
        do {
          ++e;
        } while (pre[e + 1] == pre[e]);
      }
      __syncwarp();
      if (turn) {
        const KvEntry t = kv_entry<SPARSE>(p, e, RT, U, false);
        if (lane == 0) s_ent[warp] = t;
      }
      if (lane == 0) sp.e = e, sp.h = h;
      __syncwarp();
      begin();
    }
  }
}

// Units before each entry when there are more entries than a CTA scans by itself: one CTA.
template <bool SPARSE>
__global__ void __launch_bounds__(256) kv_scan_kernel(AttendArgs p, int RT, int U) {
  __shared__ long long s_warp[8];
  __shared__ int s_wcnt[8];
  pdl_wait();
  pdl_trigger();
  kv_scan<SPARSE, 8>(p, RT, U, true, s_warp, s_wcnt, p.prefix, p.count, nullptr, nullptr);
}

// Joins the parts of the query rows that were cut between workers, in the workers' order, and writes the
// rows that see no key: o = sum_i 2^(lse_i - max) o_i / sum_i 2^(lse_i - max).  WPR warps share a row:
// eight where few rows are cut into many parts, one where there are many rows.  It is a chain of loads,
// so each step's loads are issued together: the row's place from the batch's own arrays before the
// parts are waited for, then four parts with their logsumexps at a time.
constexpr int kJoinThreads = 256;
constexpr unsigned int kJoinScanCtas = 2 * 148;  // (with 4 x 148 the last of a larger grid scan too late: drafts 21.3 -> 22.3 us)
template <int HD, bool SPARSE, int WPR>
__global__ void __launch_bounds__(kJoinThreads) kv_join_kernel(AttendArgs p, int RT, int U, int rows) {
  constexpr int V = HD / 32;  // dims of a lane
  constexpr int W = kJoinThreads / 32;
  __shared__ float s_m[W], s_l[W];
  __shared__ float s_o[W][HD];
  __shared__ long long s_pre[kScanSmem + 1], s_warp[W];
  __shared__ int s_cnt[kScanSmem + 1], s_wcnt[W];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp % WPR;
  const int row = blockIdx.x * (W / WPR) + warp / WPR;
  const int seg = p.by_rv(row), n = row - seg * p.RV;
  const int e = p.by_hkv(seg), h = seg - e * p.Hkv;
  // The batch's arrays are older than the kernel before this one, which has waited for them.  A grid of one
  // wave scans them again meanwhile; a larger one reads what that kernel has left (loads on its critical path).
  KvEntry t;
  t.nrows = 0;
  if (row < rows) t = kv_entry<SPARSE>(p, e, RT, U, false);
  const bool scan = !p.scanned && gridDim.x <= kJoinScanCtas;
  bool mine = n < t.nrows;
  long long w0 = 0, w1 = -1;
  auto locate = [&](const long long* pre, const int* cnt) {
    if (mine && t.nrec > 0) {
      const long long total = (pre[p.E] + (long long)kSegWeight * cnt[p.E]) * p.Hkv;
      const long long workers = min((long long)p.max_workers, total);
      const long long at =
          (pre[e] + (long long)kSegWeight * cnt[e]) * p.Hkv + (long long)h * (t.nrec + kSegWeight) + kSegWeight;
      w0 = worker_of(at, total, workers);
      w1 = worker_of(at + t.nrec - 1, total, workers);
      mine = w0 != w1;  // else one worker had all of it
    }
  };
  if (scan) {
    kv_scan<SPARSE, W>(p, RT, U, false, s_warp, s_wcnt, s_pre, s_cnt, nullptr, nullptr);
    locate(s_pre, s_cnt);
  }
  pdl_wait();
  pdl_trigger();
  if (SPARSE && blockIdx.x == 0) kv_report_bad(p.rows, p.ctl, 9);
  if (!scan) locate(p.prefix, p.count);
  if (!mine && WPR == 1) return;
  if (WPR == W && !mine) return;  // the whole block
  float acc[V], sum = 0.f, mx = -INFINITY;
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.f;
  for (long long w = w0 + sub; mine && w <= w1; w += 4 * WPR) {
    float ls[4], v[4][V];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const long long wk = w + k * WPR;
      const bool live = wk <= w1;
      // the first worker's part is its last (slot 1), the others' their first (slot 0)
      const long long r = (wk * 2 + (wk == w0 ? 1 : 0)) * p.RV + n;
      ls[k] = live ? p.part_lse[r] : -INFINITY;
      const float* src = p.part_o + r * HD + lane * V;
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        const float2 f = live ? *reinterpret_cast<const float2*>(src + i) : make_float2(0.f, 0.f);
        v[k][i] = f.x, v[k][i + 1] = f.y;
      }
    }
    const float m4 = fmaxf(fmaxf(mx, fmaxf(ls[0], ls[1])), fmaxf(ls[2], ls[3]));
    const float ref = m4 == -INFINITY ? 0.f : m4;
    const float f = ex2_approx(mx - ref);
    mx = m4;
    sum *= f;
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] *= f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float g = ex2_approx(ls[k] - ref);
      sum += g;
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] += g * v[k][i];
    }
  }
  if (WPR > 1) {
#pragma unroll
    for (int i = 0; i < V; ++i) s_o[warp][lane * V + i] = acc[i];
    if (lane == 0) s_m[warp] = mx, s_l[warp] = sum;
    __syncthreads();
    if (!mine || sub != 0) return;
    mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < WPR; ++i) mx = fmaxf(mx, s_m[warp + i]);
    const float ref = mx == -INFINITY ? 0.f : mx;
    sum = 0.f;
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] = 0.f;
#pragma unroll
    for (int i = 0; i < WPR; ++i) {
      const float g = ex2_approx(s_m[warp + i] - ref);
      sum += s_l[warp + i] * g;
#pragma unroll
      for (int k = 0; k < V; ++k) acc[k] += s_o[warp + i][lane * V + k] * g;
    }
  }
  const float ref = mx == -INFINITY ? 0.f : mx;
  const int rho = t.rho0 + n, tok = p.by_g(rho);
  const long long qrow = (long long)(t.row0 + tok) * p.H + h * p.G + rho - tok * p.G;
  const float f = sum == 0.f ? 0.f : 1.f / sum;
  __nv_bfloat16* out = p.o + qrow * HD + lane * V;
#pragma unroll
  for (int i = 0; i < V; i += 2)
    *reinterpret_cast<__nv_bfloat162*>(out + i) = __floats2bfloat162_rn(acc[i] * f, acc[i + 1] * f);
  if (lane == 0 && p.lse) p.lse[qrow] = sum == 0.f ? -INFINITY : (ref + log2f(sum)) * 0.6931471805599453f;
}

// ------------------------------------------------------------------ host

struct AttendPlan {
  int NT, QC, RT, QT, RV;
  long long E;
  size_t count_off, lse_off, o_off, total;
};

static int attend_plan(const char* what, const gpt_kv_cache* c, const gpt_kv_batch* b, int M, int H, int sparse,
                       AttendPlan* out) {
  const std::string w(what);
  if (H < 1 || H % c->n_kv_head) return set_error(ST_INVALID_ARG, w + ": H must be a multiple of n_kv_head");
  const long long G = H / c->n_kv_head;
  const long long max_new = kv_max_new(b);
  const long long rows = sparse ? G : max_new * G;  // query rows of a sequence (sparse: of a token) and kv head
  AttendPlan p;
  // Query rows of a tile: 4, 8 or 16 by the rows there are.  Measured at 9 to 16 rows and more (8 bits,
  // heads of 64 and 128): tiles of 16 are 4 to 25 % faster than tiles of 8, which read the cache twice as
  // often, but for very small batches (13.4 us against 11.1).
  p.NT = rows <= 8 ? 1 : 2;
  p.QC = rows <= 4 ? 1 : 2;
  p.RT = 4 * p.NT * p.QC;
  const long long qt = rows > 0 ? (rows + p.RT - 1) / p.RT : 0;
  p.RV = (int)(rows < p.RT ? (rows > 0 ? rows : 1) : p.RT);
  p.E = (sparse ? (long long)M : (long long)b->n_seq) * qt;
  if (qt > 0x7fffffffLL || p.E > 0x7fffffffLL / ((long long)c->n_kv_head * p.RV))  // (the product may pass 2^63)
    return set_error(ST_UNSUPPORTED, w + ": too many query rows");
  p.QT = (int)qt;
  auto al = [](size_t x) { return (x + 255) & ~size_t(255); };
  p.count_off = al((size_t)(p.E + 1) * 8);
  p.lse_off = p.count_off + al((size_t)(p.E + 1) * 4);
  p.o_off = p.lse_off + al((size_t)kAttendMaxWorkers * 2 * p.RV * 4);
  p.total = p.o_off + (size_t)kAttendMaxWorkers * 2 * p.RV * c->head_dim * 4;
  *out = p;
  return ST_OK;
}

template <class G, int NT, int QC, bool SPARSE>
static int launch_attend(AttendArgs a, const AttendPlan& pl, double bytes, double flops, cudaStream_t st) {
  using C = AttendCfg<G, NT>;
  auto kern = kv_attend_kernel<G, NT, QC, SPARSE>;
  static bool attr_set[64] = {};
  int dev = 0;
  GPTK_CUDA(cudaGetDevice(&dev));
  if (!attr_set[dev & 63]) {
    GPTK_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM));
    attr_set[dev & 63] = true;
  }
  int grid = num_sms() * C::CTAS;
  if (grid > kAttendMaxWorkers / C::WARPS) grid = kAttendMaxWorkers / C::WARPS;
  a.max_workers = grid * C::WARPS;
  a.worker_m = ~0ULL / a.max_workers + 1;
  if (a.scanned) {
    Prof prof(PK_ATTN_FWD, 0, 0, st);
    GPTK_CUDA(launch_pdl(kv_scan_kernel<SPARSE>, dim3(1), dim3(256), 0, st, a, pl.RT, (int)C::U));
  }
  {
    Prof prof(PK_ATTN_FWD, flops, bytes, st);
    GPTK_CUDA(launch_pdl(kern, dim3(grid), dim3(C::WARPS * 32), C::SMEM, st, a));
  }
  // warps a row of the join: by the parts that a row has on average when every worker is busy (with eight, two
  // and one; 8 bits, lengths to 4096: 4 x 10 heads, 44 parts, 13.1 / 16.0 / 19.4 us; 24 x 2 heads of 16 rows, 25 parts,
  // 21.9 / 25.3 / 29.2; 48 of them, 12 parts, 32.1 / 30.2 / 32.5; 80, 7 parts, 46 / 39.9 / 41; 32 x 10 heads of one row,
  // 5.5 parts, 57 / 57 / 53)
  const long long segs = pl.E * a.Hkv, workers = (long long)grid * C::WARPS;
  const long long parts = workers / segs;
  const int rows = (int)(segs * pl.RV);
  Prof prof(PK_ATTN_FWD, 0, 0, st);
  auto join = [&](auto kern, int wpr) {
    const unsigned int per = kJoinThreads / 32 / wpr;
    return launch_pdl(kern, dim3((rows + per - 1) / per), dim3(kJoinThreads), 0, st, a, pl.RT, (int)C::U, rows);
  };
  GPTK_CUDA(parts >= 24  ? join(kv_join_kernel<G::HD, SPARSE, 8>, 8)
            : parts >= 6 ? join(kv_join_kernel<G::HD, SPARSE, 2>, 2)
                         : join(kv_join_kernel<G::HD, SPARSE, 1>, 1));
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
  size_t block_bytes = 0;
  GPTK_TRY(kv_dispatch(cache, [&](auto g) {
    block_bytes = (size_t)decltype(g)::TILE * cache->n_kv_head;
    return (int)ST_OK;
  }));
  if (block_bytes > 0x7fffffff) return set_error(ST_UNSUPPORTED, "attention_kv: a block's tiles above 2 GiB");
  if ((long long)batch->n_seq * batch->max_blocks > 0x7fffffffLL)
    return set_error(ST_UNSUPPORTED, "attention_kv: block table above 2^31 entries");
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
  a.n_blocks = cache->n_blocks;
  a.block_bytes = (unsigned int)block_bytes;
  a.H = H;
  a.Hkv = cache->n_kv_head;
  a.G = H / cache->n_kv_head;
  a.n_sel = n_sel;
  a.window = window;
  a.E = (int)pl.E;
  a.QT = pl.QT;
  a.RV = pl.RV;
  a.by_qt = KvDiv(a.QT), a.by_g = KvDiv(a.G), a.by_rv = KvDiv(a.RV), a.by_hkv = KvDiv(a.Hkv);
  a.scanned = pl.E > kScanSmem;
  a.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)cache->head_dim));
  a.o = static_cast<__nv_bfloat16*>(o);
  a.lse = lse;
  char* sp = static_cast<char*>(scratch);
  a.prefix = reinterpret_cast<long long*>(sp);
  a.count = reinterpret_cast<int*>(sp + pl.count_off);
  a.part_lse = reinterpret_cast<float*>(sp + pl.lse_off);
  a.part_o = reinterpret_cast<float*>(sp + pl.o_off);
  a.ctl = device_ctl();
  if (!a.ctl.status) return set_error(ST_CUDA, "device status word unavailable");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return kv_dispatch(cache, [&](auto g) -> int {
    using G = decltype(g);
    if (n_sel > 0) {
      if (pl.QC == 1) return launch_attend<G, 1, 1, true>(a, pl, 0, 0, st);
      if (pl.NT == 1) return launch_attend<G, 1, 2, true>(a, pl, 0, 0, st);
      return launch_attend<G, 2, 2, true>(a, pl, 0, 0, st);
    }
    if (pl.QC == 1) return launch_attend<G, 1, 1, false>(a, pl, 0, 0, st);
    if (pl.NT == 1) return launch_attend<G, 1, 2, false>(a, pl, 0, 0, st);
    return launch_attend<G, 2, 2, false>(a, pl, 0, 0, st);
  });
}

}  // extern "C"
