// latent_attend.cu -- attention of every head over a paged cache of latent rows, the
// absorbed form (sm_103a).
//
//   out[t][h] = sum_k p_k c_k,   p = softmax_k scale q[t][h] . [c_k | r_k]
// The cache row of a key, [c (dc) | r (dr)], is key and (its first dc elements)
// value of all heads at once, so a request's rows are (token, head) pairs and a
// key's row serves all of them from shared memory.
//
// Per key and head 2 (2 dc + dr) flops against 2 (dc + dr) bytes per key: at dc =
// 512 the balance of HBM and tensor cores is near 128 heads.  A CTA holds R = 16,
// 32 or 64 rows and walks tiles of 48 or 64 keys.  One copy of a tile in shared memory
// feeds both MMAs of tcgen05:
//   S (64 x keys) = Q K^T, M the rows, K-major; M = 64 leaves S's rows on the first
//     16 lanes of each warp;
//   O^T (128 dims x R, dc / 128 of them) += V^T P^T, M the dims (the same bytes
//     read MN-major), N the rows.  O transposed keeps all 128 lanes busy for any R
//     and takes dc / 128 * R <= 256 TMEM columns (O itself would take all 512).
// P goes through shared memory as the B operand, in the cache's type, which is all
// that the MMA takes beside 16-bit values; the normaliser sums it in fp32 before that.
// (bf16: 2.0e-3 from the result in 64 bits in root mean square, relative; 1.7e-3 with P
// in fp32, which is the rounding of the result alone.  f16, long contexts: 2.1e-4 both.)
//
// An MMA costs its issue 34 to 40 cycles however few keys it has, so S (36 of them
// for 576 dims) wants large tiles, and the copies want several tiles in flight: a
// tile's slot is empty from its P V until its next copy, some 2000 cycles of HBM and 1500
// of softmax later.  Beside up to 32 rows of Q three tiles of 48 keys fit, beside 64
// rows two of 64.  (8 x 125 k keys, 32 heads: 200 us with two of 64, 208 with five of 32,
// 192 so; 64 requests, 128 heads: 90 with two of 64, 92 with four of 32.)
//
// Measured: 8 x 125 k keys on 32 heads 188 us, 6.1 TB/s; 64 requests of 512 to 4096 keys
// on 16 heads 44 (25 for the bytes: the start takes some 10 us and the merge 6), on
// 128 heads 83; 24 chunks beside 40 single tokens on 32 heads 225 us, 565 TFLOP/s.  The
// last two are bound by a slot's life, with two of them: copy 1550 to 2000 cycles, S
// 1310 (2100 beside a P V), softmax 1100 and P into shared memory 640 with the waits,
// P V 690 to 1200.  (Eight softmax warps on half of the keys each were no faster: 85 and
// 229 us beside 84 and 227.)
//
// A tile lies as [8 keys][64-element column block][8 x 128 bytes], so that the rows
// of a page land with one copy whatever the block size: a copy holds its warp for
// some 200 ns.
//
// Work: the batch's (row tile, key tile) grid, row tile after row tile, is cut into
// equal shares, one per CTA (fewer where a share would be below LEAST_SHARE
// tiles).  A row tile cut by a share's border leaves unnormalised partials with
// their max and sum, which a second kernel merges in a fixed order.  In a batch of
// single tokens with more than 64 heads, the CTAs of a share work side by side
// on the row tiles of one token, so HBM is read once for all of them (when this was
// chosen: 64 requests on 128 heads 87 us, 94 with a share each; on 256 heads 142 and 156).
//
// Eight warps: 0-3 softmax and epilogue, 4 and 6 TMA of the cache, 5 TMA of Q and the
// MMAs of S, 7 the MMAs of P V.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstddef>

#include "../../include/pattn.h"
#include "common.cuh"
#include "internal.h"

namespace pattn {
namespace {

constexpr int LA_THREADS = 256;
// Keys of a tile (above): three tiles of 48 in the ring, or two of 64 beside 64 rows.
__host__ __device__ constexpr int la_keys(int R) { return R == 64 ? 64 : 48; }
constexpr int PAD = 2;                // a row tile's fixed cost, in key tiles
constexpr int LEAST_SHARE = 3;        // cost of a CTA's share, in key tiles
constexpr int LA_BOX = 16;            // cache rows of a copy (runs of 32 took as long)
constexpr int LA_AHEAD = 1;           // tiles asked for in L2 before their copies
constexpr float LA_RESCALE_LOG2 = 8.f;
constexpr int LA_MOST_KEYS = 0x7fffff00;  // of a request: 32 bits hold a few tiles more
constexpr unsigned FULL = 0xffffffffu;
constexpr int MAX_SHARES = 160;  // (the merge keeps their weights in shared memory)

// Where a share begins: key tile t of row tile j of request r, with the request as
// la_request gives it (so that a CTA's first copies wait for one load less).
struct __align__(16) Cut {
  int r, j, t, known;
  int t0, q, s, pad;
};

struct LaHeader {
  unsigned status;  // written by the merge: the CTAs' own words together
  int shares;  // written by the attention's first CTA, for the merge
  int pad[62];
};
static_assert(sizeof(LaHeader) == 256 && offsetof(LaHeader, status) == offsetof(WsHeader, status),
              "the status word is where pattn_read_device_status looks for it");

struct LaProblem {
  const int* block_table;
  const int* seq_lens;
  const int* qsl;
  uint16_t* out;
  LaHeader* hdr;
  unsigned* cta_status;  // [grid]
  Cut* cuts;        // [shares + 1]
  float* part_o;    // [grid][2][R / 4][dc][4]: what a CTA's first and last row tile leave
  float2* part_ml;  // [grid][2][R]: their max (log2 units) and sum
  float sl2;
  int B, T, H, dc, dr, bs, mbps, NB, causal, half;
  int R, r_shift;   // rows of a row tile, a power of two
  int keys;         // of a key tile
  int lanes;        // CTAs side by side on a share (1, or the row tiles of a token)
  int max_shares;
  int fused;        // rotary parts of 64 elements: copied with the latents
  int test_skip;    // wait-test build only
};

// A request's rows and keys; false (and the rows clipped to out) if they are bad.
__device__ __forceinline__ bool la_request(const LaProblem& p, int r, int& t0, int& q, int& s) {
  t0 = p.qsl[r];
  q = p.qsl[r + 1] - t0;
  s = p.seq_lens[r];
  if (q == 0) return true;
  if (q > 0 && s >= q && s <= static_cast<int64_t>(p.mbps) * p.bs && s <= LA_MOST_KEYS && t0 >= 0 &&
      q <= p.T - t0 && (p.lanes == 1 || q == 1))
    return true;
  const int64_t end = static_cast<int64_t>(t0) + q;
  t0 = min(max(t0, 0), p.T);
  q = static_cast<int>(max(static_cast<int64_t>(0), min(end, static_cast<int64_t>(p.T)) - t0));
  s = 0;
  return false;
}

// (A call has fewer than 2^31 (token, head) rows.)
__device__ __forceinline__ int la_row_tiles(const LaProblem& p, int q) {
  if (p.lanes > 1) return q > 0 ? 1 : 0;  // (a lane's own)
  return static_cast<int>((static_cast<unsigned>(q) * static_cast<unsigned>(p.H) + p.R - 1) >> p.r_shift);
}

// Key tiles of row tile j (a bad request's counts one, in which nothing is done).
__device__ __forceinline__ int la_key_tiles(const LaProblem& p, int q, int s, int j) {
  if (s == 0) return 1;
  int keys = s;
  if (p.causal && q > 1) {
    const unsigned last = (static_cast<unsigned>(j + 1) << p.r_shift) - 1;
    keys = s - q + min(q - 1, static_cast<int>(last / static_cast<unsigned>(p.H))) + 1;
  }
  return (keys + p.keys - 1) / p.keys;
}

// The cost of a request's first x row tiles, a x + b x^2 / 2: the key tiles grow
// with the position.  (An estimate where rows and tiles do not divide; it only
// says where the shares are cut.  Two CTAs compute the cut between them, each for
// itself, so every product and sum below is rounded as it stands: 0.5 b and the
// differences of counts are exact, the rest is spelled out.)
struct Cost {
  float a, b;
  int n;  // row tiles
};
__device__ __forceinline__ Cost la_cost(const LaProblem& p, int q, int s) {
  Cost c;
  c.n = la_row_tiles(p, q);
  c.a = static_cast<float>(la_key_tiles(p, q, s, 0) + PAD);
  c.b = 0.f;
  if (c.n > 1) {
    c.b = (static_cast<float>(la_key_tiles(p, q, s, c.n - 1) + PAD) - c.a) / static_cast<float>(c.n - 1);
    c.a -= 0.5f * c.b;  // (so that n row tiles cost their sum)
  }
  return c;
}
__device__ __forceinline__ unsigned long long la_total(const LaProblem& p, int q, int s) {
  const Cost c = la_cost(p, q, s);
  const float n = static_cast<float>(c.n);
  return static_cast<unsigned long long>(rintf(__fmul_rn(n, __fmaf_rn(0.5f * c.b, n, c.a))));
}

// ------------------------------------------------------------------- plan

// The sum of x over the CTA's threads before this one, and over all of them.
__device__ __forceinline__ unsigned long long sum_before(unsigned long long x,
                                                         unsigned long long* warp_sums,
                                                         unsigned long long& all) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  unsigned long long incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long y = __shfl_up_sync(FULL, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();  // (the sums of the last use have been read)
  if (lane == 31) warp_sums[wid] = incl;
  __syncthreads();
  unsigned long long before = 0ull;
  all = 0ull;
#pragma unroll
  for (int w = 0; w < LA_THREADS / 32; ++w) {
    const unsigned long long y = warp_sums[w];
    if (w < wid) before += y;
    all += y;
  }
  return before + incl - x;
}

// Where weight w of request r falls, v past the request's begin.
__device__ __forceinline__ Cut la_place(const LaProblem& p, int r, int t0, int q, int s, float v) {
  const Cost k = la_cost(p, q, s);
  const float root = __fsqrt_rn(fmaxf(0.f, __fmaf_rn(k.a, k.a, __fmul_rn(2.f * k.b, v))));
  const float x = 2.f * v / __fadd_rn(k.a, root);
  Cut cut = {r, min(static_cast<int>(x), k.n - 1), 0, 1, t0, q, s, 0};
  const int nk = la_key_tiles(p, q, s, cut.j);
  cut.t = static_cast<int>(__fmul_rn(x - static_cast<float>(cut.j), static_cast<float>(nk + PAD)));
  if (cut.t >= nk) {  // behind the row tile's keys: the next one begins
    cut.t = 0;
    if (++cut.j >= k.n) cut = {r + 1, 0, 0, 0, 0, 0, 0, 0};
  }
  return cut;
}

// Cuts the batch into shares: every CTA sums the requests' costs (integers, so that all
// agree) and finds the two cuts of its share; the first one leaves all of them for the
// merge.  (When this was chosen a kernel of its own before them took as long, 50.1 us for
// 64 requests on 16 heads against 50.3 without it, and it is a launch more.)
__device__ __forceinline__ void la_plan(const LaProblem& p, int share, unsigned long long* warp_sums,
                                        Cut* mine, int* shares_out, unsigned* status) {
  const int tid = threadIdx.x;
  int t0_0 = 0, q_0 = 0, s_0 = 0;  // request tid, for both passes
  unsigned long long x_0 = 0ull, sum = 0ull, total;
  bool bad = false;
  for (int r = tid; r < p.B; r += LA_THREADS) {
    int t0, q, s;
    bad |= !la_request(p, r, t0, q, s);
    const unsigned long long x = la_total(p, q, s);
    sum += x;
    if (r == tid) {
      t0_0 = t0;
      q_0 = q;
      s_0 = s;
      x_0 = x;
    }
  }
  unsigned long long before = sum_before(sum, warp_sums, total);
  const int shares = static_cast<int>(
      max(1ull, min(static_cast<unsigned long long>(p.max_shares), total / LEAST_SHARE)));
  const bool first = blockIdx.x == 0;
  if (tid == 0) {
    *shares_out = shares;
    mine[0] = {0, 0, 0, 0, 0, 0, 0, 0};
    mine[1] = {p.B, 0, 0, 0, 0, 0, 0, 0};
  }
  __syncthreads();
  if (first) {
    if (bad) flag_status(status, PATTN_DEV_BAD_METADATA);
    if (tid == 0) {
      p.hdr->shares = shares;
      p.cuts[0] = {0, 0, 0, 0, 0, 0, 0, 0};
      p.cuts[shares] = {p.B, 0, 0, 0, 0, 0, 0, 0};
    }
  }
  // Pass 2: the request that weight total * c / shares falls into.
  auto weight = [&](int c) { return total * static_cast<unsigned>(c) / static_cast<unsigned>(shares); };
  unsigned long long done = 0ull;
  for (int base = 0; base < p.B; base += LA_THREADS) {
    const int r = base + tid;
    int t0 = t0_0, q = q_0, s = s_0;
    unsigned long long x = x_0, all;
    if (base > 0) {
      x = 0ull;
      if (r < p.B) {
        la_request(p, r, t0, q, s);
        x = la_total(p, q, s);
      }
    }
    if (p.B > LA_THREADS) before = sum_before(x, warp_sums, all) + done;
    if (x > 0ull) {
      if (first) {
        for (int c = max(1, static_cast<int>(before * shares / total)); c < shares; ++c) {
          const unsigned long long w = weight(c);
          if (w >= before + x) break;
          if (w < before) continue;
          p.cuts[c] = la_place(p, r, t0, q, s, static_cast<float>(w - before));
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int c = share + e;
        if (c < 1 || c >= shares) continue;
        const unsigned long long w = weight(c);
        if (w >= before && w < before + x)
          mine[e] = la_place(p, r, t0, q, s, static_cast<float>(w - before));
      }
    }
    if (p.B > LA_THREADS) done += all;
  }
  __syncthreads();
}

// ------------------------------------------------------------------ the walk

// A CTA's part of one row tile.
struct Seg {
  int r, j;
  int t0, q, s;     // the request's first row, rows and keys (0: bad, write zeros)
  int k0, k1, nk;   // key tiles, of nk
  int64_t row0;     // first (token, head) row, in q's and out's rows
  int rows;
};

struct Walk {
  Cut at, end;
};

// The next part, or false.  lane: which row tile of a token (lanes > 1).
__device__ __forceinline__ bool la_next(const LaProblem& p, Walk& w, int lane, Seg& g) {
  for (;;) {
    if (w.at.r >= p.B) return false;
    if (w.at.r == w.end.r && w.at.j == w.end.j && w.at.t >= w.end.t) return false;
    if (w.at.r > w.end.r || (w.at.r == w.end.r && w.at.j > w.end.j)) return false;
    if (!w.at.known) {
      la_request(p, w.at.r, w.at.t0, w.at.q, w.at.s);
      w.at.known = 1;
    }
    g.t0 = w.at.t0;
    g.q = w.at.q;
    g.s = w.at.s;
    if (w.at.j >= la_row_tiles(p, g.q)) {
      w.at = {w.at.r + 1, 0, 0, 0, 0, 0, 0, 0};
      continue;
    }
    g.r = w.at.r;
    g.j = w.at.j;
    g.nk = la_key_tiles(p, g.q, g.s, g.j);
    g.k0 = w.at.t;
    g.k1 = (w.end.r == g.r && w.end.j == g.j) ? w.end.t : g.nk;
    const int64_t first = static_cast<int64_t>(p.lanes > 1 ? lane : g.j) * p.R;
    const int64_t all = static_cast<int64_t>(g.q) * p.H;
    g.row0 = static_cast<int64_t>(g.t0) * p.H + first;
    g.rows = static_cast<int>(min(static_cast<int64_t>(p.R), all - first));
    // (a bad request may have more rows than the lanes of a single token)
    if (g.s == 0 && p.lanes > 1) g.rows = lane == 0 ? static_cast<int>(all) : 0;
    w.at.t = 0;
    ++w.at.j;
    if (g.k1 < g.nk) w.at = w.end;
    if (p.lanes > 1 && g.rows <= 0) continue;
    return true;
  }
}

// ------------------------------------------------------------------ attention

template <int R>
struct LaCfg {
  static constexpr int QBLK = R * 128;         // a 64-element column block of Q
  static constexpr int KEYS = la_keys(R);
  static constexpr int NST = R == 64 ? 2 : 3;  // tiles in the ring
  static constexpr int ROT = KEYS * 128;       // bytes of a tile's rotary parts
  static constexpr int LAT = 8 * ROT;          // and of its latents (dc = 512)
  static constexpr int STAGE = LAT + ROT;
  static constexpr int Q_OFF = 0;
  static constexpr int P_OFF = Q_OFF + 9 * QBLK;
  static constexpr int K_OFF = P_OFF + R * 128;
  static constexpr int BAR_OFF = K_OFF + NST * STAGE;
  static constexpr int SMEM = BAR_OFF + 1024 + 1024;
  static_assert(SMEM <= 232448, "a CTA's shared memory");
  static_assert(P_OFF % 1024 == 0 && K_OFF % 1024 == 0, "swizzled blocks are 1024-byte aligned");
  static constexpr int EC = R < 32 ? R : 32;   // columns of O that the epilogue takes at once
  static constexpr unsigned S_COL = 256;       // two score buffers of 64 columns
};

struct LaBars {
  uint64_t k_full[3], k_empty[3][2];  // (a slot's two copying warps are let in apart)
  uint64_t q_full, q_empty, s_full[2], s_empty[2], p_full, pv_done, drain[2];
  float alpha[64], l[64];
  Cut cuts[2];
  unsigned long long sums[LA_THREADS / 32];
  int shares;
  unsigned status;  // of this CTA
  unsigned tmem_base;
  int abort_flag;
};
static_assert(sizeof(LaBars) <= 1024, "the barriers fit the space kept for them");

// 16 TMEM lanes x 64 fp32 columns of a warp: lane t gets columns 8 g + 2 (t % 4) + {0,
// 1} of rows t / 4 (v[4 g], v[4 g + 1]) and t / 4 + 8 (v[4 g + 2], v[4 g + 3]).
__device__ __forceinline__ void tc_ld_scores(unsigned taddr, float (&v)[32]) {
  unsigned* r = reinterpret_cast<unsigned*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
        "=r"(r[31])
      : "r"(taddr));
}

// The same for 48 columns, with the last 16 from a copy of their own.
__device__ __forceinline__ void tc_ld_scores(unsigned taddr, float (&v)[24]) {
  unsigned* r = reinterpret_cast<unsigned*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
      : "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
        "=r"(r[22]), "=r"(r[23])
      : "r"(taddr + 32));
}

// 16 consecutive fp32 columns of this thread's TMEM lane.
__device__ __forceinline__ void tc_ld16(unsigned taddr, float (&v)[16]) {
  unsigned* r = reinterpret_cast<unsigned*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

__device__ __forceinline__ void tc_ld_cols(unsigned taddr, float (&v)[16]) { tc_ld16(taddr, v); }
__device__ __forceinline__ void tc_ld_cols(unsigned taddr, float (&v)[32]) { tc_ld32(taddr, v); }

// Barrier 1 over the softmax threads; whether any of them asked.
__device__ __forceinline__ bool any_of_128(bool ask) {
  unsigned r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 q, %1, 0;\n\t"
      "bar.red.or.pred p, 1, 128, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(static_cast<unsigned>(ask))
      : "memory");
  return r != 0;
}

template <int R, bool HALF>
__global__ void __launch_bounds__(LA_THREADS, 1)
    latent_kernel(const __grid_constant__ LaProblem p, const __grid_constant__ CUtensorMap qmap,
                  const __grid_constant__ CUtensorMap cmap,
                  const __grid_constant__ CUtensorMap rmap,
                  const __grid_constant__ CUtensorMap qrmap) {
  using C = LaCfg<R>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  LaBars* bars = reinterpret_cast<LaBars*>(smem + C::BAR_OFF);
  unsigned* status = &bars->status;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NST; ++i) {
      mbar_init(&bars->k_full[i], 2);  // the latents' and the rotary parts' bytes
      mbar_init(&bars->k_empty[i][0], 1);
      mbar_init(&bars->k_empty[i][1], 1);
    }
    mbar_init(&bars->q_full, 1);
    mbar_init(&bars->q_empty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->s_full[i], 1);
      mbar_init(&bars->s_empty[i], 4);  // read by a softmax warp
      mbar_init(&bars->drain[i], 1);
    }
    mbar_init(&bars->p_full, 128);
    mbar_init(&bars->pv_done, 1);
    bars->abort_flag = 0;
    bars->status = 0u;
    fence_mbar_init();
    tma_prefetch_desc(&qmap);
    tma_prefetch_desc(&cmap);
    if (!p.fused) {
      tma_prefetch_desc(&rmap);
      tma_prefetch_desc(&qrmap);
    }
  }
  if (warp == 0) {
    tmem_alloc(&bars->tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const unsigned tmem = bars->tmem_base;
  volatile int* abort_flag = &bars->abort_flag;
  const int share = blockIdx.x / p.lanes, side = blockIdx.x % p.lanes;
  grid_dep_trigger();  // (with the TMEM in hand, which a later kernel's CTA could take)
  grid_dep_wait();
  la_plan(p, share, bars->sums, bars->cuts, &bars->shares, status);
  const bool works = share < bars->shares;
  unsigned char* sQ = smem + C::Q_OFF;
  unsigned char* sP = smem + C::P_OFF;
  unsigned char* sK = smem + C::K_OFF;
  const int nc = p.dc / 64;  // column blocks of the latents
  const int cols = nc + p.fused;  // of a copied row
  const int nd = p.dc / 128;
  constexpr int ppt = C::KEYS / LA_BOX;  // pages of a tile
  const int first = p.fused ? (ppt + 1) / 2 : ppt;  // of which warp 4 copies these

  if (!works) {
  } else if (warp == 4 || warp == 6) {
    // ---------------------------------------------------------------- TMA
    // Rotary parts of 64 elements come with the latents, a copy a page, and warps 4 and
    // 6 have half of the pages each (a copy holds its warp for some 200 ns); others come
    // through a map that widens them with zeros, copied by warp 6.  Lane 0 waits for
    // a ring slot and posts its warp's bytes, the copies go out from one lane each.
    const int half = warp == 6 ? 1 : 0;
    const bool rot = !p.fused && half;
    Walk w = {bars->cuts[0], bars->cuts[1]};
    Seg g;
    int pos = 0, ok = 1;
#ifdef PATTN_WAIT_TEST
    // wait-test build: this tile's first half posts no bytes and issues no copy
    const int skip_pos = (p.test_skip == 3 && half == 0 && blockIdx.x == 0) ? 0 : -1;
#else
    constexpr int skip_pos = -1;
#endif
    const int page = (p.fused && half ? first : 0) + lane;  // this lane's
    const int last = half ? ppt : first;
    const int page_bytes = rot ? LA_BOX * 128 : LA_BOX * 128 * cols;
    while (ok && la_next(p, w, side, g)) {
      if (g.s == 0) continue;
      const int* bt = p.block_table + static_cast<int64_t>(g.r) * p.mbps;
      // the pool row that the lane's page of key tile kt begins at, -1 for none
      auto page_row = [&](int kt) {
        const int key = kt * C::KEYS + page * LA_BOX;
        if (page >= last || kt >= g.k1 || key >= g.s) return -1;
        int blk = bt[key / p.bs];
        if (blk < 0 || blk >= p.NB) {
          flag_status(status, PATTN_DEV_BAD_METADATA);
          blk = min(max(blk, 0), p.NB - 1);
        }
        return blk * p.bs + key % p.bs;
      };
      // Tiles past the ring are asked for in L2: two tiles in flight do not cover the
      // latency of HBM.
      int rows[LA_AHEAD + 1];
      auto ask = [&](int row) {
        if (row < 0) return;
        if (rot) tma_prefetch_3d(&rmap, 0, 0, row >> 3);
        else tma_prefetch_4d(&cmap, 0, 0, 0, row >> 3);
      };
#pragma unroll
      for (int e = 0; e <= LA_AHEAD; ++e) {
        rows[e] = page_row(g.k0 + e);
        if (e > 0) ask(rows[e]);
      }
      for (int kt = g.k0; kt < g.k1; ++kt, ++pos) {
        const int row = rows[0], st = pos % C::NST;
#pragma unroll
        for (int e = 0; e < LA_AHEAD; ++e) rows[e] = rows[e + 1];
        rows[LA_AHEAD] = page_row(kt + 1 + LA_AHEAD);
        if (pos == skip_pos) continue;
        const int copies = __popc(__ballot_sync(FULL, row >= 0));
        if (lane == 0) {
          if (pos >= C::NST &&
              !mbar_wait(&bars->k_empty[st][half], ((pos / C::NST) - 1) & 1, status, abort_flag))
            ok = 0;
          else if (copies > 0)
            mbar_arrive_expect_tx(&bars->k_full[st], static_cast<unsigned>(copies * page_bytes));
          else
            mbar_arrive(&bars->k_full[st]);
        }
        ok = __shfl_sync(FULL, ok, 0);
        if (!ok) break;
        if (row >= 0) {
          unsigned char* dst = sK + st * C::STAGE + (rot ? C::LAT : 0) + page * page_bytes;
          if (rot)
            tma_load_3d(dst, &rmap, &bars->k_full[st], 0, 0, row >> 3);
          else
            tma_load_4d(dst, &cmap, &bars->k_full[st], 0, 0, 0, row >> 3);
        }
        ask(rows[LA_AHEAD]);
      }
    }
    // A role gave up on a wait: no copy may still be writing shared memory when the
    // CTA exits.  (A slot's phase also needs the other producer's bytes; if that one
    // gave up first, this wait runs out instead.)
    if ((!ok || *abort_flag) && lane == 0) {
      drain_armed(bars->k_full, C::NST, pos, skip_pos, status);
    }
    __syncwarp();
  } else if (warp == 5 || warp == 7) {
    // ---------------------------------------------------------------- MMA
    // S and P V have a warp each.  The whole warp walks, with every value that the
    // descriptors are made of the same in all lanes and known to be (reductions over
    // the warp), and the elected lane issues: an MMA of S then takes 34 cycles (M 64, N
    // 64; its operands take 32 to read).  With lane 0 in place of the elected one it
    // took 54, from a branch for one lane 46 to 71.
    const bool scores = warp == 5;
    const unsigned lead = elect_one();
    constexpr unsigned idesc_s = make_idesc_f16(64, C::KEYS, !HALF, false);
    constexpr unsigned idesc_pv = make_idesc_f16(128, R, !HALF, false) | (1u << 15);  // A MN-major
    const unsigned t_base = __reduce_max_sync(FULL, tmem);
    const uint64_t q_d = smem_desc_sw128(smem_u32(sQ), 16, 1024);
    const uint64_t p_d = smem_desc_sw128(smem_u32(sP), 16, 1024);
    // 8 keys are `cols` KB apart; of V, 64 dims are 1 KB apart
    const uint64_t k_d = smem_desc_sw128(smem_u32(sK), 16, cols * 1024);
    const uint64_t r_d = smem_desc_sw128(smem_u32(sK + (p.fused ? nc * 1024 : C::LAT)), 16,
                                         p.fused ? cols * 1024 : 1024);
    const uint64_t v_d = smem_desc_sw128(smem_u32(sK), 1024, cols * 1024);
    Walk w = {bars->cuts[0], bars->cuts[1]};
    Seg g;
    int n = 0, n_seg = 0;  // tile of the CTA, parts of row tiles
    bool ok = true;
    while (ok && __reduce_max_sync(FULL, static_cast<unsigned>(la_next(p, w, side, g)))) {
      const int n_tiles = static_cast<int>(
          __reduce_max_sync(FULL, g.s == 0 ? 0u : static_cast<unsigned>(g.k1 - g.k0)));
      if (n_tiles == 0) continue;
      if (scores) {
        // Q, once the scores of the part before are done
        if (n_seg > 0 &&
            !__all_sync(FULL, mbar_wait(&bars->q_empty, (n_seg - 1) & 1, status, abort_flag)))
          break;
        if (lead) {
          mbar_arrive_expect_tx(&bars->q_full, static_cast<unsigned>((nc + 1) * C::QBLK));
          tma_load_3d(sQ, &qmap, &bars->q_full, 0, static_cast<int>(g.row0), 0);
          if (!p.fused)
            tma_load_3d(sQ + nc * C::QBLK, &qrmap, &bars->q_full, 0, static_cast<int>(g.row0), 0);
        }
        ++n_seg;
        if (!__all_sync(FULL, mbar_wait(&bars->q_full, (n_seg - 1) & 1, status, abort_flag))) break;
      }
      for (int i = 0; i < n_tiles; ++i, ++n) {
        const int st = n % C::NST;
        if (scores) {
          bool there = n < 2 || mbar_wait(&bars->s_empty[n & 1], ((n >> 1) - 1) & 1, status,
                                          abort_flag);
          there = there && mbar_wait(&bars->k_full[st], (n / C::NST) & 1, status, abort_flag);
          if (!__all_sync(FULL, there)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const unsigned s_t = t_base + C::S_COL + (n & 1) * 64;
          uint64_t qb = q_d, kb = k_d + ((st * C::STAGE) >> 4);
          for (int d = 0; d < nd; ++d) {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              tc_mma_ss_if(lead, s_t, qb + (((kk >> 2) * C::QBLK + (kk & 3) * 32) >> 4),
                           kb + (((kk >> 2) * 1024 + (kk & 3) * 32) >> 4), idesc_s,
                           (kk > 0 || d > 0) ? 1u : 0u);
            qb += (2 * C::QBLK) >> 4;
            kb += 2048 >> 4;
          }
          kb = r_d + ((st * C::STAGE) >> 4);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            if (kk < p.dr / 16)
              tc_mma_ss_if(lead, s_t, qb + ((kk * 32) >> 4), kb + ((kk * 32) >> 4), idesc_s, 1u);
          if (lead) {
            tc_commit(&bars->s_full[n & 1]);
            if (i == n_tiles - 1) tc_commit(&bars->q_empty);
          }
        } else {
          if (!__all_sync(FULL, mbar_wait(&bars->p_full, n & 1, status, abort_flag))) {
            ok = false;
            break;
          }
          tc_fence_after();
          uint64_t vb = v_d + ((st * C::STAGE) >> 4), pb = p_d;
          for (int kk = 0; kk < C::KEYS / 16; ++kk) {
#pragma unroll
            for (int d = 0; d < 4; ++d)
              if (d < nd)
                tc_mma_ss_if(lead, t_base + d * R, vb + ((d * 2048) >> 4), pb, idesc_pv,
                             (i > 0 || kk > 0) ? 1u : 0u);
            vb += (2 * cols * 1024) >> 4;
            pb += 32 >> 4;
            if (lead && (kk + 1) * 16 == first * LA_BOX) tc_commit(&bars->k_empty[st][0]);
          }
          if (lead) {
            tc_commit(&bars->k_empty[st][1]);
            tc_commit(&bars->pv_done);
          }
        }
      }
    }
    // no MMA may still be running when TMEM is released (matters only when a role gave
    // up on a wait)
    if (lead) {
      uint64_t* drain = &bars->drain[scores ? 0 : 1];
      tc_commit(drain);
      mbar_wait(drain, 0, status, nullptr);
      // (nor may Q's copy be in flight)
      if (n_seg > 0) mbar_wait(&bars->q_full, (n_seg - 1) & 1, status, nullptr);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax
    // Warp w's TMEM lanes 32 w .. + 15 hold rows 16 w .. + 15 of S; a thread has two
    // of them, ra and ra + 8, and a quarter of the keys of each.
    const bool has_rows = warp * 16 < R;
    const int ra = warp * 16 + (lane >> 2), c2 = 2 * (lane & 3);
    const unsigned lane_base = tmem + (static_cast<unsigned>(warp * 32) << 16);
    const float sl2 = p.sl2;
    int tile = 0;
    bool ok = true;
    Walk w = {bars->cuts[0], bars->cuts[1]};
    Seg g;
    while (la_next(p, w, side, g)) {
      uint16_t* out = p.out + g.row0 * p.dc;
      if (g.s == 0) {  // a bad request's rows
        for (int64_t e = threadIdx.x; e < static_cast<int64_t>(g.rows) * p.dc / 8; e += 128)
          reinterpret_cast<uint4*>(out)[e] = make_uint4(0u, 0u, 0u, 0u);
        continue;
      }
      // row i of the tile sees keys below kmax
      int kmax[2] = {g.s, g.s}, first_max = g.s;
      if (p.causal && g.q > 1) {
        const unsigned in_req = static_cast<unsigned>(g.row0 - static_cast<int64_t>(g.t0) * p.H);
        const unsigned H = static_cast<unsigned>(p.H);
        first_max = g.s - g.q + static_cast<int>(in_req / H) + 1;
#pragma unroll
        for (int e = 0; e < 2; ++e)
          kmax[e] = min(g.s, g.s - g.q + static_cast<int>((in_req + ra + 8 * e) / H) + 1);
      }
      float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
      const int n_tiles = g.k1 - g.k0;
      for (int i = 0; i < n_tiles; ++i) {
        const int n = tile + i, key0 = (g.k0 + i) * C::KEYS;
        if (!__all_sync(FULL, mbar_wait(&bars->s_full[n & 1], (n >> 1) & 1, status, abort_flag)))
          ok = false;
        float v[C::KEYS / 2];
        bool ask = false;
        float alpha[2] = {1.f, 1.f};
        if (ok && has_rows) {
          tc_fence_after();
          tc_ld_scores(lane_base + C::S_COL + (n & 1) * 64, v);
          tc_wait_ld();
          tc_fence_before();
          if (lane == 0) mbar_arrive(&bars->s_empty[n & 1]);
          if (key0 + C::KEYS > first_max) {
#pragma unroll
            for (int e = 0; e < C::KEYS / 2; ++e) {
              const int key = key0 + (e >> 2) * 8 + c2 + (e & 1);
              if (key >= kmax[(e >> 1) & 1]) v[e] = -INFINITY;
            }
          }
          float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int e = 0; e < C::KEYS / 2; ++e) mx[(e >> 1) & 1] = fmaxf(mx[(e >> 1) & 1], v[e]);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            mx[e] = fmaxf(mx[e], __shfl_xor_sync(FULL, mx[e], 1));
            mx[e] = fmaxf(mx[e], __shfl_xor_sync(FULL, mx[e], 2));
            const float x = mx[e] == -INFINITY ? -INFINITY : mx[e] * sl2;
            // the reference moves only where the max grows by more than 2^8
            if (x > m[e] + LA_RESCALE_LOG2 || (m[e] == -INFINITY && x > m[e])) {
              if (m[e] != -INFINITY) {
                alpha[e] = fast_exp2(m[e] - x);
                l[e] *= alpha[e];
                ask = true;
              }
              m[e] = x;
            }
          }
#pragma unroll
          for (int e = 0; e < C::KEYS / 2; ++e) {
            const int k = (e >> 1) & 1;
            v[e] = fast_exp2(v[e] * sl2 - (m[k] == -INFINITY ? 0.f : m[k]));
            l[k] += v[e];
          }
        }
        if (!has_rows && lane == 0) mbar_arrive(&bars->s_empty[n & 1]);
        const bool rescale = any_of_128(ask);
        // P V of the tile before has read P, and O may be rescaled
        if (ok && n > 0 &&
            !__all_sync(FULL, mbar_wait(&bars->pv_done, (n - 1) & 1, status, abort_flag)))
          ok = false;
        if (rescale) {
          if (has_rows && (lane & 3) == 0) {
            bars->alpha[ra] = alpha[0];
            bars->alpha[ra + 8] = alpha[1];
          }
          named_bar_sync(1, 128);
          if (ok) {
            tc_fence_after();
            for (int d = 0; d < nd; ++d)
#pragma unroll
              for (int c = 0; c < R; c += 16) {
                float o[16];
                tc_ld16(lane_base + d * R + c, o);
                tc_wait_ld();
                unsigned u[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) u[e] = __float_as_uint(o[e] * bars->alpha[c + e]);
                tc_st16u(lane_base + d * R + c, u);
              }
            tc_wait_st();
          }
        }
        if (!ok) continue;  // (the barriers of the loop stay matched)
        if (has_rows) {
#pragma unroll
          for (int c = 0; c < C::KEYS / 8; ++c)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int row = ra + 8 * e;
              *reinterpret_cast<unsigned*>(sP + row * 128 + ((c ^ (row & 7)) << 4) + c2 * 2) =
                  pack2<HALF>(v[4 * c + 2 * e], v[4 * c + 2 * e + 1]);
            }
        }
        // Values of keys at or past seq_len become zero before P V reads them: the
        // slots may hold anything, and 0 * NaN is NaN.
        const int tail = g.s - key0;
        if (tail < C::KEYS) {
          unsigned char* k = sK + (n % C::NST) * C::STAGE;
          const int x = threadIdx.x & 63;  // 16-byte piece of a row
          if (x < 8 * nc)
            for (int row = tail + (threadIdx.x >> 6); row < C::KEYS; row += 2)
              *reinterpret_cast<uint4*>(k + ((row >> 3) * cols + (x >> 3)) * 1024 + (row & 7) * 128 +
                                        (x & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(&bars->p_full);
      }
      tile += n_tiles;
      // --------------------------------------------------------- epilogue
      // All of the row tile's keys: normalised rows to out.  A part of them: sums,
      // their reference max and their weights' sum to the CTA's first or second
      // partial (of a row tile begun in an earlier share; of one begun here).
      const bool whole = n_tiles == g.nk;
      const int64_t part = static_cast<int64_t>(blockIdx.x) * 2 + (g.k0 > 0 ? 0 : 1);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[e] += __shfl_xor_sync(FULL, l[e], 1);
        l[e] += __shfl_xor_sync(FULL, l[e], 2);
        if (has_rows && (lane & 3) == 0) {
          if (whole)
            bars->l[ra + 8 * e] = l[e] > 0.f ? 1.f / l[e] : l[e] == 0.f ? 0.f : NAN;
          else
            p.part_ml[part * R + ra + 8 * e] = make_float2(m[e], l[e]);
        }
      }
      if (ok && !__all_sync(FULL, mbar_wait(&bars->pv_done, (tile - 1) & 1, status, abort_flag)))
        ok = false;
      if (any_of_128(!ok)) break;  // (all four warps, so that none waits for another)
      tc_fence_after();
      // Lane: a dim of the block; columns: the rows.
      if (!whole) {
        float4* po = reinterpret_cast<float4*>(p.part_o) + part * (R / 4) * p.dc + warp * 32 + lane;
        for (int d = 0; d < nd; ++d, po += 128)
#pragma unroll
          for (int c = 0; c < R; c += C::EC) {
            if (c >= g.rows) break;
            float o[C::EC];
            tc_ld_cols(lane_base + d * R + c, o);
            tc_wait_ld();
#pragma unroll
            for (int e = 0; e < C::EC; e += 4)
              po[static_cast<int64_t>((c + e) / 4) * p.dc] = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
          }
      } else {
        // neighbouring lanes swap rows, so that each writes two dims of one row
        const int odd = lane & 1;
        uint16_t* ob = out + warp * 32 + (lane & ~1) + static_cast<int64_t>(odd) * p.dc;
        for (int d = 0; d < nd; ++d, ob += 128)
#pragma unroll
          for (int c = 0; c < R; c += C::EC) {
            if (c >= g.rows) break;
            float o[C::EC];
            tc_ld_cols(lane_base + d * R + c, o);
            tc_wait_ld();
            // (the stores last: behind one, the next weight's load and exchange would wait)
            unsigned w[C::EC / 2];
#pragma unroll
            for (int e = 0; e < C::EC; ++e) o[e] *= bars->l[c + e];
#pragma unroll
            for (int e = 0; e < C::EC; e += 2) {
              const float got = __shfl_xor_sync(FULL, odd ? o[e] : o[e + 1], 1);
              w[e / 2] = odd ? pack2<HALF>(got, o[e + 1]) : pack2<HALF>(o[e], got);
            }
            uint16_t* row = ob + static_cast<int64_t>(c) * p.dc;
#pragma unroll
            for (int e = 0; e < C::EC; e += 2, row += 2 * p.dc)
              if (c + e + odd < g.rows) *reinterpret_cast<unsigned*>(row) = w[e / 2];
          }
      }
      tc_fence_before();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0) p.cta_status[blockIdx.x] = bars->status;
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// --------------------------------------------------------------------- merge

// CTA (x, y): rows 8 G y .. of the row tile that the CTA x of the attention began and
// left to the next shares, if it did.  The parts' weights come first (a warp a row, its
// lanes the parts), under the loads of the sums; a thread then adds up a dim of 4 G
// rows.  Bound by latency: the parts were written long ago and come from HBM.
template <bool HALF, int G>
__global__ void __launch_bounds__(1024) latent_merge_kernel(const __grid_constant__ LaProblem p) {
  constexpr int U = 8 / G;  // parts in flight
  constexpr int ROWS = 8 * G;
  __shared__ float weight[MAX_SHARES][ROWS];
  grid_dep_trigger();
  grid_dep_wait();
  const int share = blockIdx.x / p.lanes, side = blockIdx.x % p.lanes;
  const int tid = threadIdx.x, lane = tid & 31;
  if (blockIdx.x + 1 == gridDim.x && blockIdx.y == 0 && tid < 32) {
    unsigned any = 0u;
    for (unsigned i = lane; i < gridDim.x; i += 32) any |= p.cta_status[i];
    any = __reduce_or_sync(FULL, any);
    if (lane == 0) p.hdr->status = any;
  }
  const int shares = p.hdr->shares;
  // lane i: the cut i shares on
  const int4* cuts = reinterpret_cast<const int4*>(p.cuts);
  const int mine = min(share + lane, p.max_shares);
  const int4 c = cuts[2 * mine], c1 = cuts[2 * mine + 1];
  if (share + 1 >= shares) return;
  const int4 a = {__shfl_sync(FULL, c.x, 0), __shfl_sync(FULL, c.y, 0), __shfl_sync(FULL, c.z, 0), 0};
  const int4 b = {__shfl_sync(FULL, c.x, 1), __shfl_sync(FULL, c.y, 1), __shfl_sync(FULL, c.z, 1), 0};
  const int t0 = __shfl_sync(FULL, c1.x, 1), q = __shfl_sync(FULL, c1.y, 1);
  if (b.z == 0 || (a.x == b.x && a.y == b.y && a.z > 0)) return;
  // (a cut inside a row tile knows its request, which is not a bad one)
  const int64_t first = static_cast<int64_t>(p.lanes > 1 ? side : b.y) * p.R;
  const int rows = static_cast<int>(min(static_cast<int64_t>(p.R),
                                        static_cast<int64_t>(q) * p.H - first));
  const int row0 = blockIdx.y * ROWS;
  if (row0 >= rows) return;
  // shares that hold a part of it: the cuts behind this share that lie inside it
  auto inside = [&](int i, const int4& k) {
    return i < shares && k.x == b.x && k.y == b.y && k.z > 0;
  };
  unsigned off = ~(__ballot_sync(FULL, inside(share + lane, c)) | 3u);
  int parts = off ? __ffs(off) - 1 : 32;
  while (!off) {
    const int i = min(share + parts + lane, p.max_shares);
    off = ~__ballot_sync(FULL, share + parts + lane < shares && inside(i, cuts[2 * i]));
    parts += off ? __ffs(off) - 1 : 32;
  }
  // part i's place: the second partial of the first share, the first of the others
  auto at = [&](int i) {
    return static_cast<int64_t>((share + i) * p.lanes + side) * 2 + (i == 0 ? 1 : 0);
  };
  const int dim = tid % p.dc, group0 = row0 / 4 + tid / p.dc * G;  // the thread's row groups
  float4 x[U][G];
  auto load = [&](int i0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float4* s = reinterpret_cast<const float4*>(p.part_o) +
                        (at(min(i0 + u, parts - 1)) * (p.R / 4) + group0) * p.dc + dim;
#pragma unroll
      for (int g = 0; g < G; ++g) x[u][g] = s[static_cast<int64_t>(g) * p.dc];
    }
  };
  load(0);
#pragma unroll 1
  for (int row = tid >> 5; row < ROWS; row += blockDim.x >> 5) {
    const float2* ml = p.part_ml + row0 + row;
    float top = -INFINITY;
#pragma unroll 1
    for (int i = lane; i < parts; i += 32) top = fmaxf(top, ml[at(i) * p.R].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(FULL, top, o));
    const float ref = top == -INFINITY ? 0.f : top;
    float l = 0.f;
#pragma unroll 1
    for (int i = lane; i < parts; i += 32) {
      const float2 v = ml[at(i) * p.R];
      const float w = fast_exp2(v.x - ref);
      weight[i][row] = w;
      l += w * v.y;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(FULL, l, o);
    const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : NAN;
#pragma unroll 1
    for (int i = lane; i < parts; i += 32) weight[i][row] *= inv;
  }
  __syncthreads();
  float4 acc[G];
#pragma unroll
  for (int g = 0; g < G; ++g) acc[g] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int i0 = 0; i0 < parts; i0 += U) {
    if (i0 > 0) load(i0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i0 + u >= parts) break;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const float4 w = *reinterpret_cast<const float4*>(&weight[i0 + u][(group0 + g) * 4 - row0]);
        acc[g].x += w.x * x[u][g].x;
        acc[g].y += w.y * x[u][g].y;
        acc[g].z += w.z * x[u][g].z;
        acc[g].w += w.w * x[u][g].w;
      }
    }
  }
  uint16_t* out = p.out + (static_cast<int64_t>(t0) * p.H + first) * p.dc + dim;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const float v[4] = {acc[g].x, acc[g].y, acc[g].z, acc[g].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int row = (group0 + g) * 4 + e;
      if (row < rows)
        out[static_cast<int64_t>(row) * p.dc] = static_cast<uint16_t>(pack2<HALF>(v[e], 0.f));
    }
  }
}

// ---------------------------------------------------------------------- host

// Row tile: 64 rows, or what a request's rows need where that is less.
int la_rows(int max_q, int H) {
  const long long rows = static_cast<long long>(max_q) * H;
  return rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
}

struct LaLayout {
  size_t status, cuts, ml, o, total;
  int grid;
};
LaLayout la_layout(int dc) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  LaLayout l;
  l.grid = std::min(current_sms(), MAX_SHARES);
  l.status = sizeof(LaHeader);
  l.cuts = up(l.status + sizeof(unsigned) * l.grid);
  l.ml = up(l.cuts + sizeof(Cut) * (l.grid + 1));
  l.o = up(l.ml + sizeof(float2) * l.grid * 2 * 64);
  l.total = up(l.o + sizeof(float) * l.grid * 2 * 64 * dc);
  return l;
}

template <int R, bool HALF>
cudaError_t launch_latent(const LaProblem& p, const CUtensorMap (&m)[4], int grid, cudaStream_t st) {
  using C = LaCfg<R>;
  auto kern = latent_kernel<R, HALF>;
  static std::atomic<unsigned long long> ready{0};  // devices whose limit is set
  cudaError_t e = cudaErrorInvalidValue;
  for (int again = 0; again < 2 && e == cudaErrorInvalidValue; ++again) {
    e = allow_shared_memory(reinterpret_cast<const void*>(kern), C::SMEM, ready, again);
    if (e != cudaSuccess) return e;
    e = launch_dependent(kern, dim3(static_cast<unsigned>(grid)), LA_THREADS, C::SMEM, st, p, m[0],
                         m[1], m[2], m[3]);
    if (e == cudaErrorInvalidValue) cudaGetLastError();
  }
  if (e != cudaSuccess) return e;
  // a quarter as many row tiles as SMs and more: most of them in two parts, a CTA or
  // two each; else finer.  (64 requests on 128 heads: 13 us so, 26 with 8 rows a CTA
  // and 19 with 64, whose code and registers outgrow an SM.)
  constexpr int G = R >= 32 ? 4 : 2;
  const bool many = static_cast<long long>(p.B) * p.lanes * 4 >= grid;
  const dim3 ctas(static_cast<unsigned>(grid), many ? R / (8 * G) : R / 8);
  return many ? launch_dependent(latent_merge_kernel<HALF, G>, ctas, 2u * p.dc, 0, st, p)
              : launch_dependent(latent_merge_kernel<HALF, 1>, ctas, 2u * p.dc, 0, st, p);
}

template <int R>
cudaError_t launch_latent_rows(const LaProblem& p, const CUtensorMap (&m)[4], int grid, cudaStream_t st) {
  return p.half ? launch_latent<R, true>(p, m, grid, st)
                : launch_latent<R, false>(p, m, grid, st);
}

}  // namespace
}  // namespace pattn

using namespace pattn;

extern "C" size_t pattn_latent_workspace_bytes(int num_seqs, int num_heads, int latent_size) {
  if (num_seqs < 0 || num_heads <= 0 || latent_size <= 0 || latent_size % 128 != 0 ||
      latent_size > 512)
    return 0;
  return la_layout(latent_size).total;
}

extern "C" pattn_status_t pattn_latent_fwd(const pattn_latent_t* a) {
  if (!a || a->struct_size < sizeof(pattn_latent_t)) return PATTN_ERR_INVALID_ARGUMENT;
  const pattn_status_t v =
      check_latent_sizes(a->latent_size, a->rope_size, a->block_size, a->kv_dtype);
  if (v != PATTN_OK) return v;
  if (!a->q || !a->kv_cache || !a->out || !a->block_table || !a->seq_lens || !a->query_start_loc ||
      !a->workspace)
    return PATTN_ERR_INVALID_ARGUMENT;
  if (a->num_seqs < 0 || a->num_tokens < 0 || a->num_heads <= 0 || a->max_blocks_per_seq < 0 ||
      a->num_blocks < 0 || a->max_query_len < 0)
    return PATTN_ERR_INVALID_ARGUMENT;
  if (!(a->scale >= 0.f) || std::isinf(a->scale) || (a->causal != 0 && a->causal != 1))
    return PATTN_ERR_INVALID_ARGUMENT;
  for (const void* x : {a->q, a->kv_cache, static_cast<const void*>(a->out)})
    if (reinterpret_cast<uintptr_t>(x) & 15) return PATTN_ERR_INVALID_ARGUMENT;
  if (reinterpret_cast<uintptr_t>(a->workspace) & 255) return PATTN_ERR_INVALID_ARGUMENT;
  // rows and slots are counted in 32 bits by the copies
  if (static_cast<long long>(a->num_tokens) * a->num_heads > 0x7fffff00LL ||
      static_cast<long long>(a->num_blocks) * a->block_size > 0x7fffff00LL)
    return PATTN_ERR_UNSUPPORTED;
  const LaLayout l = la_layout(a->latent_size);
  if (a->workspace_bytes < l.total) return PATTN_ERR_WORKSPACE_TOO_SMALL;
  if (a->num_seqs == 0 || a->num_tokens == 0) return PATTN_OK;
  if (a->num_blocks == 0 || a->max_blocks_per_seq == 0) return PATTN_ERR_INVALID_ARGUMENT;
  const int R = la_rows(std::max(1, a->max_query_len), a->num_heads);
  LaProblem p = {};
  p.block_table = a->block_table;
  p.seq_lens = a->seq_lens;
  p.qsl = a->query_start_loc;
  p.out = static_cast<uint16_t*>(a->out);
  unsigned char* ws = static_cast<unsigned char*>(a->workspace);
  p.hdr = reinterpret_cast<LaHeader*>(ws);
  p.cta_status = reinterpret_cast<unsigned*>(ws + l.status);
  p.cuts = reinterpret_cast<Cut*>(ws + l.cuts);
  p.part_ml = reinterpret_cast<float2*>(ws + l.ml);
  p.part_o = reinterpret_cast<float*>(ws + l.o);
  // strictly positive, so that a masked score (-inf) always maps to weight 0; at
  // scale 0 the weights are 1 exactly
  p.sl2 = fmaxf(a->scale * LOG2E, 1e-30f);
  p.B = a->num_seqs;
  p.T = a->num_tokens;
  p.H = a->num_heads;
  p.dc = a->latent_size;
  p.dr = a->rope_size;
  p.bs = a->block_size;
  p.mbps = a->max_blocks_per_seq;
  p.NB = a->num_blocks;
  p.causal = a->causal;
  p.half = a->kv_dtype == PATTN_KV_F16;
  p.R = R;
  p.keys = la_keys(R);
  p.r_shift = R == 16 ? 4 : R == 32 ? 5 : 6;
  const int tiles = (a->num_heads + R - 1) / R;  // row tiles of a token
  p.lanes = a->max_query_len <= 1 && tiles > 1 && tiles <= 8 ? tiles : 1;
  p.max_shares = std::max(1, l.grid / p.lanes);
  p.fused = a->rope_size == 64;
#ifdef PATTN_WAIT_TEST
  p.test_skip = test_wait_skip();
#endif
  CUtensorMap m[4];
  if (!encode_latent_maps(m, a->q, a->kv_cache, p.half, a->latent_size, a->rope_size,
                          a->num_tokens * a->num_heads, R, a->num_blocks * a->block_size, LA_BOX))
    return PATTN_ERR_CUDA;
  const int grid = p.max_shares * p.lanes;
  cudaStream_t st = static_cast<cudaStream_t>(a->stream);
  const cudaError_t e = R == 16   ? launch_latent_rows<16>(p, m, grid, st)
                        : R == 32 ? launch_latent_rows<32>(p, m, grid, st)
                                  : launch_latent_rows<64>(p, m, grid, st);
  return e == cudaSuccess ? PATTN_OK : PATTN_ERR_CUDA;
}
