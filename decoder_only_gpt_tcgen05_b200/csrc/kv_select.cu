// Choosing the cache blocks that a query attends to: a cheap score for every visible block, then the
// n best of them.
//
// The score of block j for a token and kv head is an upper bound of what its keys can reach,
//
//   score_j = sum over the kv head's query heads g and dims d of max(q_gd kmin_jd, q_gd kmax_jd),
//
// from the elementwise bounds that the append keeps.  It is summed in fp64 and rounded once to fp32:
// the choice hangs on comparisons of near scores, and a sum in fp32 would let the order of the
// additions decide.  Equal scores go to the lower index.
//
// Measured, scores and choice together: 7.0 us for one sequence of 8k tokens (12 heads of 64: two launches and
// four dependent loads), 13.9 us for 16 of 4k to 32k (10 heads of 128, 23 MB of bounds), 18.5 us for 64 rows of 16
// heads over 2 kv heads.  Alone and with a cold cache the scores take 5.8, 12.5 and 16.7 us, the choice 6.2, 7.5 and 6.2.
// The grouped scores are bound by the conversions to fp64 (their pipe is busy for 52 % of the time, the fp64 products'
// for 13 %) and by rows of uneven length (0.26 to 0.82 instructions a clock and scheduler, by SM); the choice by its
// barriers (0.15 instructions a clock and scheduler).
#include <string>

#include "kv.cuh"

namespace gptk {

constexpr int kScoreThreads = 256;
constexpr int kScoreChunk = 64;  // blocks a CTA scores: two turns, whose loads are issued together

// One CTA: one token, one kv head, kScoreChunk blocks.  Eight lanes take a block, 16-byte pieces of
// both bounds each.  Reads 4 HD bytes a block.  ONE: one query head a kv head.  Loops stay rolled
// where they can: the CTAs are short, and fetching code that runs once costs more than it saves.  The conversions
// to fp64 run at an eighth of the fp32 rate: one a dim where a kv head has one query head (the bound is
// chosen first), two where several share them.
template <int HD, bool ONE>
__global__ void __launch_bounds__(kScoreThreads)
kv_score_kernel(const __nv_bfloat16* q, KvRows rows, const __nv_bfloat16* bounds,
                int n_blocks, int G, int Hkv, float* scores, DevCtl ctl) {
  constexpr int NC = HD / 64;
  extern __shared__ double s_q[];  // [G][NC][8 dims of a piece][8 lanes]
  __shared__ int s_phys[kScoreChunk];
  pdl_wait();  // (no early trigger: the next kernel's shared memory would leave these loads next to no L1)
  if (blockIdx.x == 0 && blockIdx.y == 0) kv_report_bad(rows, ctl, 5);
  const int m = blockIdx.x / Hkv, h = blockIdx.x - m * Hkv;
  for (int x = threadIdx.x; x < G * HD; x += kScoreThreads) {
    const int g = x / HD, d = x - g * HD;
    const float v = __bfloat162float(q[((long long)m * Hkv + h) * G * HD + x]);
    s_q[((g * NC + d / 64) * 8 + d % 8) * 8 + (d / 8) % 8] = (double)v;
  }
  const KvRow row = kv_find_row(rows, m);
  if (row.b < 0) return;
  const int nb = row.pos / kKvBlock + 1;
  const int j0 = blockIdx.y * kScoreChunk, j1 = min(j0 + kScoreChunk, rows.W);
  float* out = scores + ((long long)m * Hkv + h) * rows.W;
  if (j0 >= nb) {
    for (int j = j0 + threadIdx.x; j < j1; j += kScoreThreads) out[j] = -INFINITY;
    return;
  }
  for (int j = j0 + threadIdx.x; j < j1; j += kScoreThreads) {
    int phys = j < nb ? rows.table[(long long)row.b * rows.W + j] : 0;
    if (phys < 0 || phys >= n_blocks) {
      dev_report(ctl, DEV_ERR_BAD_BATCH, 6);
      phys = -1;
    }
    s_phys[j - j0] = phys;
  }
  __syncthreads();
  const int l = threadIdx.x & 7;
  constexpr int TURN = kScoreThreads / 8, TURNS = kScoreChunk / TURN;
  uint4 lo[TURNS][NC], hi[TURNS][NC];
#pragma unroll
  for (int i = 0; i < TURNS; ++i) {
    const int j = j0 + i * TURN + (threadIdx.x >> 3);
    const bool live = j < min(j1, nb);
    const int phys = live ? max(s_phys[j - j0], 0) : 0;
    const uint4* p = reinterpret_cast<const uint4*>(bounds + ((long long)phys * Hkv + h) * 2 * HD);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      lo[i][c] = live ? p[c * 8 + l] : make_uint4(0, 0, 0, 0);
      hi[i][c] = live ? p[HD / 8 + c * 8 + l] : make_uint4(0, 0, 0, 0);
    }
  }
#pragma unroll
  for (int i = 0; i < TURNS; ++i) {
    const int j = j0 + i * TURN + (threadIdx.x >> 3);
    double acc[4] = {0.0, 0.0, 0.0, 0.0};  // four chains: the fp64 add's latency is many cycles
    // (the sign of q is read from its high word: a comparison would take the fp64 unit as well)
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const uint4 vl = lo[i][c], vh = hi[i][c];
      const unsigned int ul[4] = {vl.x, vl.y, vl.z, vl.w}, uh[4] = {vh.x, vh.y, vh.z, vh.w};
      const double* qp = s_q + c * 64 + l;
      float a[8], e[8];
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        a[x] = x & 1 ? bf16_hi(ul[x >> 1]) : bf16_lo(ul[x >> 1]);
        e[x] = x & 1 ? bf16_hi(uh[x >> 1]) : bf16_lo(uh[x >> 1]);
      }
      if (ONE) {
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const double qv = qp[x * 8];
          acc[x % 4] = fma(qv, (double)(__double2hiint(qv) >= 0 ? e[x] : a[x]), acc[x % 4]);
        }
      } else {
        double da[8], de[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) da[x] = a[x], de[x] = e[x];
#pragma unroll 1
        for (int g = 0; g < G; ++g) {
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            const double qv = qp[g * HD + x * 8];
            acc[x % 4] = fma(qv, __double2hiint(qv) >= 0 ? de[x] : da[x], acc[x % 4]);
          }
        }
      }
    }
    double sum = (acc[0] + acc[1]) + (acc[2] + acc[3]);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (j < j1 && l == 0) out[j] = j >= nb ? -INFINITY : s_phys[j - j0] < 0 ? __uint_as_float(0x7fc00000u) : (float)sum;
  }
}

// One CTA picks for one token and kv head: the first n_first and last n_last visible blocks, then the
// best scores until there are n.  A radix select over the scores' ordered bits (four histograms of
// 256) finds the n-th key; one ordered pass writes the chosen indices, ascending, ties to the lower.
constexpr int kPickThreads = 256;
constexpr int kPickKeys = 4096;  // keys kept in shared memory (more are formed anew in each pass)

__device__ __forceinline__ unsigned int pick_key(float v, int j, int nb, int n_first, int n_last) {
  if (j < n_first || j >= nb - n_last) return 0xffffffffu;
  if (v != v) return 0xfffffffeu;  // a NaN score is chosen, so that it shows in the output
  const unsigned int u = __float_as_uint(v);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kPickThreads)
kv_pick_kernel(const float* scores, KvRows rows, int Hkv, int n, int n_first, int n_last,
               int* blocks) {
  __shared__ int hist[256];
  __shared__ unsigned int s_key[kPickKeys];
  __shared__ int s_bin, s_left;
  __shared__ int wsum[kPickThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int m = blockIdx.x / Hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const KvRow row = kv_find_row(rows, m);
  if (row.b < 0) return;
  const int nb = row.pos / kKvBlock + 1;
  const float* sc = scores + (long long)blockIdx.x * rows.W;
  int* out = blocks + (long long)blockIdx.x * n;
  if (nb <= n) {
    for (int i = tid; i < n; i += kPickThreads) out[i] = i < nb ? i : -1;
    return;
  }
  const bool kept = nb <= kPickKeys;
  if (kept) {
    for (int j = tid; j < nb; j += kPickThreads) s_key[j] = pick_key(sc[j], j, nb, n_first, n_last);
  }
  auto key = [&](int j) { return kept ? s_key[j] : pick_key(sc[j], j, nb, n_first, n_last); };
  unsigned int prefix = 0, mask = 0;
  int left = n;  // still to be chosen among the keys that match the prefix
  for (int shift = 24; shift >= 0; shift -= 8) {
    hist[tid] = 0;
    __syncthreads();
    for (int j = tid; j < nb; j += kPickThreads) {
      const unsigned int k = key(j);
      if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255], 1);
    }
    __syncthreads();
    if (warp == 0) {  // bins from the top, eight a lane
      int own = 0;
#pragma unroll
      for (int x = 0; x < 8; ++x) own += hist[255 - (lane * 8 + x)];
      int incl = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      int before = incl - own;
      if (before < left && incl >= left) {
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const int cnt = hist[255 - (lane * 8 + x)];
          if (before < left && before + cnt >= left) s_bin = 255 - (lane * 8 + x), s_left = left - before;
          before += cnt;
        }
      }
    }
    __syncthreads();
    prefix |= (unsigned int)s_bin << shift;
    mask |= 255u << shift;
    left = s_left;
  }
  // keys above the n-th are chosen, of those equal to it the first `left`
  int gt = 0, eq = 0;  // before this chunk
  for (int base = 0; base < nb; base += kPickThreads) {
    const int j = base + tid;
    const unsigned int k = j < nb ? key(j) : 0u;
    const bool is_gt = j < nb && k > prefix, is_eq = j < nb && k == prefix;
    const unsigned int bg = __ballot_sync(0xffffffffu, is_gt), be = __ballot_sync(0xffffffffu, is_eq);
    __syncthreads();
    if (lane == 0) wsum[warp] = __popc(bg) | (__popc(be) << 16);
    __syncthreads();
    int g = gt, e = eq;
    for (int x = 0; x < kPickThreads / 32; ++x) {
      const int v = wsum[x];
      if (x < warp) g += v & 0xffff, e += v >> 16;
      gt += v & 0xffff, eq += v >> 16;
    }
    const unsigned int below = (1u << lane) - 1;
    g += __popc(bg & below), e += __popc(be & below);
    if (is_gt || (is_eq && e < left)) out[g + min(e, left)] = j;
  }
}

}  // namespace gptk

using namespace gptk;

extern "C" {

GPT_API int gpt_op_kv_select(const gpt_kv_cache* cache, const gpt_kv_batch* batch, const void* q, int M, int H,
                             int n_select, int n_first, int n_last, int32_t* blocks, float* scores, void* stream) {
  set_error(ST_OK, "");
  GPTK_TRY(kv_check("kv_select", cache, batch, M));
  const int Hkv = cache->n_kv_head;
  if (H < 1 || H % Hkv) return set_error(ST_INVALID_ARG, "kv_select: H must be a multiple of n_kv_head");
  const int G = H / Hkv;
  if (G > 32) return set_error(ST_UNSUPPORTED, "kv_select: more than 32 query heads a kv head");
  if (!cache->bounds) return set_error(ST_INVALID_ARG, "kv_select: the cache keeps no bounds");
  if (n_select < 1 || n_first < 0 || n_last < 0 || (long long)n_first + n_last > n_select)
    return set_error(ST_INVALID_ARG, "kv_select: n_select >= 1 and n_first + n_last <= n_select are needed");
  if ((long long)M * Hkv > 0x7fffffffLL) return set_error(ST_UNSUPPORTED, "kv_select: M x n_kv_head too large");
  const long long chunks = ((long long)batch->max_blocks + kScoreChunk - 1) / kScoreChunk;
  if (chunks > 65535) return set_error(ST_UNSUPPORTED, "kv_select: max_blocks above 64 x 65535");
  if (M == 0 || batch->n_seq == 0 || kv_max_new(batch) == 0) return ST_OK;
  if (!q || !blocks || !scores) return set_error(ST_INVALID_ARG, "kv_select: null q, blocks or scores");
  if ((reinterpret_cast<uintptr_t>(q) & 15) || (reinterpret_cast<uintptr_t>(blocks) & 3) ||
      (reinterpret_cast<uintptr_t>(scores) & 3))
    return set_error(ST_INVALID_ARG, "kv_select: q must be 16-byte, blocks and scores 4-byte aligned");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const DevCtl ctl = device_ctl();
  if (!ctl.status) return set_error(ST_CUDA, "device status word unavailable");
  const KvRows r = kv_rows(batch, M);
  const int hd = cache->head_dim;
  {
    Prof prof(PK_MISC, 0, (double)M * Hkv * batch->max_blocks * (4.0 * hd + 4), st);
    const dim3 grid((unsigned)(M * Hkv), (unsigned)chunks);
    const size_t smem = (size_t)G * hd * 8;
    auto* bp = static_cast<const __nv_bfloat16*>(cache->bounds);
    auto* qp = static_cast<const __nv_bfloat16*>(q);
    auto go = [&](auto kern) {
      return launch_pdl(kern, grid, dim3(kScoreThreads), smem, st, qp, r, bp, (int)cache->n_blocks, G, Hkv, scores,
                        ctl);
    };
    GPTK_CUDA(hd == 64 ? (G == 1 ? go(kv_score_kernel<64, true>) : go(kv_score_kernel<64, false>))
                       : (G == 1 ? go(kv_score_kernel<128, true>) : go(kv_score_kernel<128, false>)));
  }
  Prof prof(PK_MISC, 0, (double)M * Hkv * (4.0 * batch->max_blocks + 4.0 * n_select), st);
  GPTK_CUDA(launch_pdl(kv_pick_kernel, dim3((unsigned)(M * Hkv)), dim3(kPickThreads), 0, st,
                       static_cast<const float*>(scores), r, Hkv, n_select, n_first, n_last, blocks));
  return ST_OK;
}

}  // extern "C"
