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
// 32 or 64 rows and walks tiles of 64 keys.  One copy of a tile in shared memory
// feeds both MMAs of tcgen05:
//   S (64 x 64) = Q K^T, M the rows, K-major from the tile's 64-element column
//     blocks; M = 64 leaves S's rows on the first 16 lanes of each warp;
//   O^T (128 dims x R, dc / 128 of them) += V^T P^T, M the dims (the same blocks
//     read MN-major), N the rows.  O transposed keeps all 128 lanes busy for any R
//     and takes dc / 128 * R <= 256 TMEM columns (O itself would take all 512).
// P goes through shared memory as the B operand.  The tile's blocks form a ring of
// 16 KB pairs of blocks: S consumes them in order, P V frees them in order, so the
// next tile's copies go out block by block.
//
// Work: the batch's (row tile, key tile) grid, row tile after row tile, is cut into
// equal shares, one per CTA (fewer where a share would be below LEAST_SHARE
// tiles).  A row tile cut by a share's border leaves unnormalised partials with
// their max and sum, which a second kernel merges in a fixed order.  In a batch of
// single tokens with more than 64 heads, the CTAs of a share work side by side
// on the row tiles of one token, so HBM is read once for all of them.
//
// Six warps: 0-3 softmax and epilogue, 4 TMA, 5 MMA issue.
#include <algorithm>
#include <cmath>
#include <cstddef>

#include "../../include/pattn.h"
#include "common.cuh"
#include "internal.h"

namespace pattn {
namespace {

constexpr int LA_THREADS = 192;
constexpr int LA_KEYS = 64;           // keys of a tile
constexpr int LA_BLK = LA_KEYS * 128; // bytes of a 64-element column block of a tile
constexpr int PAD = 2;                // a row tile's fixed cost, in key tiles
constexpr int LEAST_SHARE = 3;        // cost of a CTA's share, in key tiles
constexpr float LA_RESCALE_LOG2 = 8.f;
constexpr unsigned FULL = 0xffffffffu;
constexpr int MAX_SHARES = 1024;

// Where a share begins: key tile t of row tile j of request r.
struct Cut {
  int r, j, t, pad;
};

struct LaHeader {
  unsigned status;
  int shares;  // written by the plan kernel
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
  Cut* cuts;        // [shares + 1]
  float* part_o;    // [grid][2][R][dc]: what a CTA's first and last row tile leave
  float2* part_ml;  // [grid][2][R]: their max (log2 units) and sum
  double* prefix;   // [B + 1] cost of the requests before
  float sl2;
  int B, T, H, dc, dr, bs, mbps, NB, causal, half;
  int R;            // rows of a row tile
  int lanes;        // CTAs side by side on a share (1, or the row tiles of a token)
  int max_shares;
  int box;          // cache rows of one copy
};

// A request's rows and keys; false (and the rows clipped to out) if they are bad.
__device__ __forceinline__ bool la_request(const LaProblem& p, int r, int& t0, int& q, int& s) {
  t0 = p.qsl[r];
  q = p.qsl[r + 1] - t0;
  s = p.seq_lens[r];
  if (q == 0) return true;
  if (q > 0 && s >= q && s <= static_cast<int64_t>(p.mbps) * p.bs && t0 >= 0 && q <= p.T - t0 &&
      (p.lanes == 1 || q == 1))
    return true;
  const int64_t end = static_cast<int64_t>(t0) + q;
  t0 = min(max(t0, 0), p.T);
  q = static_cast<int>(max(static_cast<int64_t>(0), min(end, static_cast<int64_t>(p.T)) - t0));
  s = 0;
  return false;
}

__device__ __forceinline__ int la_row_tiles(const LaProblem& p, int q) {
  if (p.lanes > 1) return q > 0 ? 1 : 0;  // (a lane's own)
  return static_cast<int>((static_cast<int64_t>(q) * p.H + p.R - 1) / p.R);
}

// Key tiles of row tile j (a bad request's counts one, in which nothing is done).
__device__ __forceinline__ int la_key_tiles(const LaProblem& p, int q, int s, int j) {
  if (s == 0) return 1;
  int keys = s;
  if (p.causal && p.lanes == 1) {
    const int64_t last = (static_cast<int64_t>(j) + 1) * p.R - 1;
    keys = s - q + static_cast<int>(min(static_cast<int64_t>(q - 1), last / p.H)) + 1;
  }
  return (keys + LA_KEYS - 1) / LA_KEYS;
}

// The cost of a request's first x row tiles, a x + b x^2 / 2: the key tiles grow
// with the position.  (An estimate where rows and tiles do not divide; it only
// says where the shares are cut.)
struct Cost {
  double a, b;
  int n;  // row tiles
  __device__ double upto(double x) const { return x * (a + 0.5 * b * x); }
};
__device__ __forceinline__ Cost la_cost(const LaProblem& p, int r) {
  int t0, q, s;
  la_request(p, r, t0, q, s);
  Cost c;
  c.n = la_row_tiles(p, q);
  c.a = la_key_tiles(p, q, s, 0) + PAD;
  c.b = c.n > 1 ? static_cast<double>(la_key_tiles(p, q, s, c.n - 1) + PAD - c.a) / (c.n - 1) : 0.;
  c.a -= 0.5 * c.b;  // (so that n row tiles cost their sum)
  return c;
}

// ------------------------------------------------------------------- plan

constexpr int LA_PLAN_THREADS = 1024;

__global__ void __launch_bounds__(LA_PLAN_THREADS)
    latent_plan_kernel(const __grid_constant__ LaProblem p) {
  __shared__ double warp_sums[32];
  __shared__ double carry;
  __shared__ unsigned bad;
  grid_dep_trigger();
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  if (tid == 0) {
    carry = 0.;
    bad = 0u;
  }
  __syncthreads();
  for (int base = 0; base < p.B; base += LA_PLAN_THREADS) {
    const int r = base + tid;
    double x = 0.;
    if (r < p.B) {
      int t0, q, s;
      if (!la_request(p, r, t0, q, s)) bad = PATTN_DEV_BAD_METADATA;
      const Cost c = la_cost(p, r);
      x = c.upto(c.n);
    }
    double incl = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double y = __shfl_up_sync(FULL, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) warp_sums[wid] = incl;
    __syncthreads();
    double before = carry;
    for (int w = 0; w < wid; ++w) before += warp_sums[w];
    if (r < p.B) p.prefix[r] = before + incl - x;
    __syncthreads();
    if (tid == LA_PLAN_THREADS - 1) carry = before + incl;
    __syncthreads();
  }
  const double total = carry;
  const int shares =
      max(1, min(p.max_shares, static_cast<int>(min(total / LEAST_SHARE, 1e6))));
  if (tid == 0) {
    p.hdr->status = bad;
    p.hdr->shares = shares;
  }
  for (int c = tid; c <= shares; c += LA_PLAN_THREADS) {
    Cut cut = {c == shares ? p.B : 0, 0, 0, 0};
    if (c > 0 && c < shares) {
      const double w = total * c / shares;
      int lo = 0, hi = p.B;  // the last request that costs begin at or before w
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.prefix[mid] <= w) lo = mid;
        else hi = mid;
      }
      const Cost k = la_cost(p, lo);
      const double v = w - p.prefix[lo];
      const double x = 2. * v / (k.a + sqrt(fmax(0., k.a * k.a + 2. * k.b * v)));
      int t0, q, s;
      la_request(p, lo, t0, q, s);
      cut.r = lo;
      cut.j = min(static_cast<int>(x), max(0, k.n - 1));
      const int nk = la_key_tiles(p, q, s, cut.j);
      cut.t = static_cast<int>((x - cut.j) * (nk + PAD));
      if (k.n == 0 || cut.t >= nk) {  // behind the row tile's keys: the next one begins
        cut.t = 0;
        if (++cut.j >= k.n) {
          cut.j = 0;
          ++cut.r;
        }
      }
    }
    p.cuts[c] = cut;
  }
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

__device__ __forceinline__ Walk la_walk(const LaProblem& p, int share) {
  return {p.cuts[share], p.cuts[share + 1]};
}

// The next part, or false.  lane: which row tile of a token (lanes > 1).
__device__ __forceinline__ bool la_next(const LaProblem& p, Walk& w, int lane, Seg& g) {
  for (;;) {
    if (w.at.r >= p.B) return false;
    if (w.at.r == w.end.r && w.at.j == w.end.j && w.at.t >= w.end.t) return false;
    if (w.at.r > w.end.r || (w.at.r == w.end.r && w.at.j > w.end.j)) return false;
    la_request(p, w.at.r, g.t0, g.q, g.s);
    if (w.at.j >= la_row_tiles(p, g.q)) {
      w.at = {w.at.r + 1, 0, 0, 0};
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
  static constexpr int ND = R == 64 ? 8 : R == 32 ? 10 : 11;  // pairs of blocks in the ring
  static constexpr int NR = R == 64 ? 2 : 3;   // rotary blocks
  static constexpr int Q_OFF = 0;
  static constexpr int P_OFF = Q_OFF + 9 * QBLK;
  static constexpr int D_OFF = P_OFF + R * 128;
  static constexpr int R_OFF = D_OFF + ND * 2 * LA_BLK;
  static constexpr int BAR_OFF = R_OFF + NR * LA_BLK;
  static constexpr int SMEM = BAR_OFF + 1024 + 1024;
  static_assert(SMEM <= 232448, "a CTA's shared memory");
  static_assert(P_OFF % 1024 == 0 && D_OFF % 1024 == 0, "swizzled blocks are 1024-byte aligned");
  static constexpr unsigned S_COL = 256;       // two score buffers of 64 columns
};

struct LaBars {
  uint64_t d_full[11], d_empty[11], r_full[3], r_empty[3];
  uint64_t q_full, q_empty, s_full[2], p_full, pv_done, drain;
  float alpha[64], l[64];
  unsigned tmem_base;
  int abort_flag;
};
static_assert(sizeof(LaBars) <= 1024, "the barriers fit the space kept for them");

// 16 TMEM lanes x 64 fp32 columns of a warp: lane t gets columns 8 g + 2 (t % 4) + {0,
// 1} of rows t / 4 (v[4 g], v[4 g + 1]) and t / 4 + 8 (v[4 g + 2], v[4 g + 3]).
__device__ __forceinline__ void tc_ld_16x64(unsigned taddr, float (&v)[32]) {
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
                  const __grid_constant__ CUtensorMap cmap) {
  using C = LaCfg<R>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  LaBars* bars = reinterpret_cast<LaBars*>(smem + C::BAR_OFF);
  unsigned* status = &p.hdr->status;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dep_trigger();

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::ND; ++i) {
      mbar_init(&bars->d_full[i], 1);
      mbar_init(&bars->d_empty[i], 1);
    }
    for (int i = 0; i < C::NR; ++i) {
      mbar_init(&bars->r_full[i], 1);
      mbar_init(&bars->r_empty[i], 1);
    }
    mbar_init(&bars->q_full, 1);
    mbar_init(&bars->q_empty, 1);
    mbar_init(&bars->s_full[0], 1);
    mbar_init(&bars->s_full[1], 1);
    mbar_init(&bars->p_full, 128);
    mbar_init(&bars->pv_done, 1);
    mbar_init(&bars->drain, 1);
    bars->abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&qmap);
    tma_prefetch_desc(&cmap);
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
  grid_dep_wait();  // the plan kernel's cuts

  const int share = blockIdx.x / p.lanes, side = blockIdx.x % p.lanes;
  const bool works = share < p.hdr->shares;
  unsigned char* sQ = smem + C::Q_OFF;
  unsigned char* sP = smem + C::P_OFF;
  unsigned char* sD = smem + C::D_OFF;
  unsigned char* sR = smem + C::R_OFF;
  const int nd = p.dc / 128;  // pairs of blocks of a tile

  if (!works) {
  } else if (warp == 4) {
    // ---------------------------------------------------------------- TMA
    // Lane 0 waits for a ring slot and posts its bytes; the copies, one per page
    // and column block, go out from one lane each.
    Walk w = la_walk(p, share);
    Seg g;
    int dpos = 0, rpos = 0, n_seg = 0, ok = 1;
    const int ppt = LA_KEYS / p.box;  // copies of a block
    const int my_pg = lane % ppt, my_col = lane / ppt;
    while (ok && la_next(p, w, side, g)) {
      if (g.s == 0) continue;
      if (lane == 0) {
        if (n_seg > 0 && !mbar_wait(&bars->q_empty, (n_seg - 1) & 1, status, abort_flag)) {
          ok = 0;
        } else {
          mbar_arrive_expect_tx(&bars->q_full, static_cast<unsigned>((2 * nd + 1) * C::QBLK));
          for (int c = 0; c <= 2 * nd; ++c)
            tma_load_3d(sQ + c * C::QBLK, &qmap, &bars->q_full, c * 64, 0, static_cast<int>(g.row0));
        }
      }
      ok = __shfl_sync(FULL, ok, 0);
      if (!ok) break;
      ++n_seg;
      const int* bt = p.block_table + static_cast<int64_t>(g.r) * p.mbps;
      // the pool row that page `my_pg` of key tile kt begins at
      auto page_row = [&](int kt) {
        const int key = kt * LA_KEYS + my_pg * p.box;
        if (kt >= g.k1 || key >= g.s) return 0;
        int blk = bt[key / p.bs];
        if (blk < 0 || blk >= p.NB) {
          flag_status(status, PATTN_DEV_BAD_METADATA);
          blk = min(max(blk, 0), p.NB - 1);
        }
        return blk * p.bs + key % p.bs;
      };
      int row_next = page_row(g.k0);
      for (int kt = g.k0; ok && kt < g.k1; ++kt) {
        const int row = row_next;
        row_next = page_row(kt + 1);
        const int pages = min(ppt, (g.s - kt * LA_KEYS + p.box - 1) / p.box);
        const unsigned bytes = static_cast<unsigned>(pages * p.box * 128);
        for (int d = 0; d <= nd; ++d) {
          const bool rot = d == nd;  // the rotary block comes last
          const int pos = rot ? rpos++ : dpos++, n = rot ? C::NR : C::ND, st = pos % n;
          uint64_t* full = rot ? &bars->r_full[st] : &bars->d_full[st];
          if (lane == 0) {
            if (pos >= n && !mbar_wait(rot ? &bars->r_empty[st] : &bars->d_empty[st],
                                       ((pos / n) - 1) & 1, status, abort_flag))
              ok = 0;
            else
              mbar_arrive_expect_tx(full, rot ? bytes : 2 * bytes);
          }
          ok = __shfl_sync(FULL, ok, 0);
          if (!ok) {
            --(rot ? rpos : dpos);
            break;
          }
          if (my_col < (rot ? 1 : 2) && my_pg < pages)
            tma_load_3d((rot ? sR + st * LA_BLK : sD + (2 * st + my_col) * LA_BLK) +
                            my_pg * p.box * 128,
                        &cmap, full, (2 * d + my_col) * 64, 0, row);
        }
      }
    }
    // A role gave up on a wait: no copy may still be writing shared memory when the
    // CTA exits.
    if ((!ok || *abort_flag) && lane == 0) {
      drain_armed(bars->d_full, C::ND, dpos, -1, status);
      drain_armed(bars->r_full, C::NR, rpos, -1, status);
      if (n_seg > 0) mbar_wait(&bars->q_full, (n_seg - 1) & 1, status, nullptr);
    }
    __syncwarp();
  } else if (warp == 5) {
    // ---------------------------------------------------------------- MMA
    if (lane == 0) {
      constexpr unsigned idesc_s = make_idesc_f16(64, LA_KEYS, !HALF, false);
      constexpr unsigned idesc_pv = make_idesc_f16(128, R, !HALF, false) | (1u << 15);  // A MN-major
      const uint64_t q_d = smem_desc_sw128(smem_u32(sQ), 16, 1024);
      const uint64_t p_d = smem_desc_sw128(smem_u32(sP), 16, 1024);
      const uint64_t k_d = smem_desc_sw128(smem_u32(sD), 16, 1024);
      const uint64_t r_d = smem_desc_sw128(smem_u32(sR), 16, 1024);
      const uint64_t v_d = smem_desc_sw128(smem_u32(sD), LA_BLK, 1024);
      Walk w = la_walk(p, share);
      Seg g;
      int tile = 0, n_seg = 0;  // of the CTA so far
      bool ok = true;
      // The scores of the CTA's tile n.
      auto scores = [&](int n) -> bool {
        const unsigned s_t = tmem + C::S_COL + (n & 1) * 64;
        for (int d = 0; d < nd; ++d) {
          const int pos = n * nd + d, st = pos % C::ND;
          if (!mbar_wait(&bars->d_full[st], (pos / C::ND) & 1, status, abort_flag)) return false;
          tc_fence_after();
          const uint64_t qb = q_d + ((2 * d * C::QBLK) >> 4), kb = k_d + ((2 * st * LA_BLK) >> 4);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            tc_mma_ss(s_t, qb + (((kk >> 2) * C::QBLK + (kk & 3) * 32) >> 4),
                      kb + (((kk >> 2) * LA_BLK + (kk & 3) * 32) >> 4), idesc_s,
                      (d > 0 || kk > 0) ? 1u : 0u);
        }
        const int st = n % C::NR;
        if (!mbar_wait(&bars->r_full[st], (n / C::NR) & 1, status, abort_flag)) return false;
        tc_fence_after();
        const uint64_t qb = q_d + ((2 * nd * C::QBLK) >> 4), kb = r_d + ((st * LA_BLK) >> 4);
        for (int kk = 0; kk < p.dr / 16; ++kk)
          tc_mma_ss(s_t, qb + ((kk * 32) >> 4), kb + ((kk * 32) >> 4), idesc_s, 1u);
        tc_commit(&bars->r_empty[st]);
        tc_commit(&bars->s_full[n & 1]);
        return true;
      };
      while (ok && la_next(p, w, side, g)) {
        if (g.s == 0) continue;
        if (!mbar_wait(&bars->q_full, n_seg & 1, status, abort_flag)) break;
        ++n_seg;
        const int n_tiles = g.k1 - g.k0;
        for (int i = 0; ok && i <= n_tiles; ++i) {
          if (i < n_tiles) {
            if (!scores(tile + i)) {
              ok = false;
              break;
            }
            if (i == n_tiles - 1) tc_commit(&bars->q_empty);
          }
          if (i == 0) continue;
          const int n = tile + i - 1;  // P V of the tile before
          if (!mbar_wait(&bars->p_full, n & 1, status, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          for (int d = 0; d < nd; ++d) {
            const int st = (n * nd + d) % C::ND;
            const uint64_t vb = v_d + ((2 * st * LA_BLK) >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              tc_mma_ss(tmem + d * R, vb + ((kk * 2048) >> 4), p_d + ((kk * 32) >> 4), idesc_pv,
                        (i > 1 || kk > 0) ? 1u : 0u);
            tc_commit(&bars->d_empty[st]);
          }
          tc_commit(&bars->pv_done);
        }
        tile += n_tiles;
      }
      // no MMA may still be running when TMEM is released (matters only when a role
      // gave up on a wait)
      tc_commit(&bars->drain);
      mbar_wait(&bars->drain, 0, status, nullptr);
    }
  } else {
    // ------------------------------------------------------------ softmax
    // Warp w's TMEM lanes 32 w .. + 15 hold rows 16 w .. + 15 of S; a thread has two
    // of them, ra and ra + 8, and 16 keys of each.
    const bool has_rows = warp * 16 < R;
    const int ra = warp * 16 + (lane >> 2), c2 = 2 * (lane & 3);
    const unsigned lane_base = tmem + (static_cast<unsigned>(warp * 32) << 16);
    const float sl2 = p.sl2;
    int tile = 0;
    bool ok = true;
    Walk w = la_walk(p, share);
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
      if (p.causal) {
        const int64_t in_req = g.row0 - static_cast<int64_t>(g.t0) * p.H;
        first_max = g.s - g.q + static_cast<int>(in_req / p.H) + 1;
#pragma unroll
        for (int e = 0; e < 2; ++e)
          kmax[e] = min(g.s, g.s - g.q + static_cast<int>((in_req + ra + 8 * e) / p.H) + 1);
      }
      float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
      const int n_tiles = g.k1 - g.k0;
      for (int i = 0; i < n_tiles; ++i) {
        const int n = tile + i, key0 = (g.k0 + i) * LA_KEYS;
        if (!__all_sync(FULL, mbar_wait(&bars->s_full[n & 1], (n >> 1) & 1, status, abort_flag)))
          ok = false;
        float v[32];
        bool ask = false;
        float alpha[2] = {1.f, 1.f};
        if (ok && has_rows) {
          tc_fence_after();
          tc_ld_16x64(lane_base + C::S_COL + (n & 1) * 64, v);
          tc_wait_ld();
          if (key0 + LA_KEYS > first_max) {
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const int key = key0 + (e >> 2) * 8 + c2 + (e & 1);
              if (key >= kmax[(e >> 1) & 1]) v[e] = -INFINITY;
            }
          }
          float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int e = 0; e < 32; ++e) mx[(e >> 1) & 1] = fmaxf(mx[(e >> 1) & 1], v[e]);
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
          for (int e = 0; e < 32; ++e) {
            const int k = (e >> 1) & 1;
            v[e] = fast_exp2(v[e] * sl2 - (m[k] == -INFINITY ? 0.f : m[k]));
            l[k] += v[e];
          }
        }
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
          for (int c = 0; c < 8; ++c)
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
        if (tail < LA_KEYS) {
          for (int e = threadIdx.x; e < (LA_KEYS - tail) * 16 * nd; e += 128) {
            const int pair = e / (16 * (LA_KEYS - tail)), x = e % (16 * (LA_KEYS - tail));
            *reinterpret_cast<uint4*>(sD + (2 * ((n * nd + pair) % C::ND) + (x & 1)) * LA_BLK +
                                      (tail + (x >> 4)) * 128 + ((x >> 1) & 7) * 16) =
                make_uint4(0u, 0u, 0u, 0u);
          }
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
      float* po = p.part_o + part * R * p.dc;
      for (int d = 0; d < nd; ++d) {
        const int dim = d * 128 + warp * 32 + lane;
#pragma unroll
        for (int c = 0; c < R; c += 16) {
          if (c >= g.rows) break;
          float o[16];
          tc_ld16(lane_base + d * R + c, o);
          tc_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            if (c + e >= g.rows) break;
            if (whole)
              out[static_cast<int64_t>(c + e) * p.dc + dim] =
                  static_cast<uint16_t>(pack2<HALF>(o[e] * bars->l[c + e], 0.f));
            else
              po[(c + e) * p.dc + dim] = o[e];
          }
        }
      }
      tc_fence_before();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// --------------------------------------------------------------------- merge

constexpr int LM_WARPS = 8;

// CTA (x, y): rows 8 y .. of the row tile that the CTA x of the attention began and
// left to the next shares, if it did.  A warp merges a row.
template <bool HALF>
__global__ void __launch_bounds__(LM_WARPS * 32)
    latent_merge_kernel(const __grid_constant__ LaProblem p) {
  grid_dep_wait();
  const int share = blockIdx.x / p.lanes, side = blockIdx.x % p.lanes;
  const int shares = p.hdr->shares;
  if (share + 1 >= shares) return;
  const Cut a = p.cuts[share], b = p.cuts[share + 1];
  if (b.t == 0 || (a.r == b.r && a.j == b.j && a.t > 0)) return;
  int parts = 2;  // shares that hold a part of it
  while (share + parts < shares) {
    const Cut c = p.cuts[share + parts];
    if (c.r != b.r || c.j != b.j || c.t == 0) break;
    ++parts;
  }
  int t0, q, s;
  if (!la_request(p, b.r, t0, q, s)) return;
  const int64_t first = static_cast<int64_t>(p.lanes > 1 ? side : b.j) * p.R;
  const int64_t rows = min(static_cast<int64_t>(p.R), static_cast<int64_t>(q) * p.H - first);
  const int row = blockIdx.y * LM_WARPS + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (row >= rows) return;
  // part i's place: the second partial of the first share, the first of the others
  auto at = [&](int i) {
    return (static_cast<int64_t>((share + i) * p.lanes + side) * 2 + (i == 0 ? 1 : 0)) * p.R + row;
  };
  float mx = -INFINITY;
  for (int i = lane; i < parts; i += 32) mx = fmaxf(mx, p.part_ml[at(i)].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, o));
  const float ref = mx == -INFINITY ? 0.f : mx;
  float4 acc[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.f;
  const int n4 = p.dc / 128;
#pragma unroll 4
  for (int i = 0; i < parts; ++i) {
    const float2 ml = p.part_ml[at(i)];
    const float wgt = fast_exp2(ml.x - ref);
    l += wgt * ml.y;
    const float4* o = reinterpret_cast<const float4*>(p.part_o + at(i) * p.dc);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < n4) {
        const float4 x = o[e * 32 + lane];
        acc[e].x += wgt * x.x;
        acc[e].y += wgt * x.y;
        acc[e].z += wgt * x.z;
        acc[e].w += wgt * x.w;
      }
  }
  const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : NAN;
  uint16_t* out = p.out + (static_cast<int64_t>(t0) * p.H + first + row) * p.dc;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < n4)
      reinterpret_cast<uint2*>(out)[e * 32 + lane] =
          make_uint2(pack2<HALF>(acc[e].x * inv, acc[e].y * inv),
                     pack2<HALF>(acc[e].z * inv, acc[e].w * inv));
}

// ---------------------------------------------------------------------- host

// Row tile: 64 rows, or what a request's rows need where that is less.
int la_rows(int max_q, int H) {
  const long long rows = static_cast<long long>(max_q) * H;
  return rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
}

struct LaLayout {
  size_t cuts, prefix, ml, o, total;
  int grid;
};
LaLayout la_layout(int B, int dc) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  LaLayout l;
  l.grid = std::min(current_sms(), MAX_SHARES);
  l.cuts = sizeof(LaHeader);
  l.prefix = up(l.cuts + sizeof(Cut) * (l.grid + 1));
  l.ml = up(l.prefix + sizeof(double) * (static_cast<size_t>(B) + 1));
  l.o = up(l.ml + sizeof(float2) * l.grid * 2 * 64);
  l.total = up(l.o + sizeof(float) * l.grid * 2 * 64 * dc);
  return l;
}

template <int R, bool HALF>
cudaError_t launch_latent(const LaProblem& p, const CUtensorMap& qmap, const CUtensorMap& cmap,
                          int grid, cudaStream_t st) {
  using C = LaCfg<R>;
  auto kern = latent_kernel<R, HALF>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  latent_plan_kernel<<<1, LA_PLAN_THREADS, 0, st>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(LA_THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, p, qmap, cmap);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(static_cast<unsigned>(grid), R / LM_WARPS);
  cfg.blockDim = dim3(LM_WARPS * 32);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, latent_merge_kernel<HALF>, p);
}

template <int R>
cudaError_t launch_latent_rows(const LaProblem& p, const CUtensorMap& qmap, const CUtensorMap& cmap,
                               int grid, cudaStream_t st) {
  return p.half ? launch_latent<R, true>(p, qmap, cmap, grid, st)
                : launch_latent<R, false>(p, qmap, cmap, grid, st);
}

}  // namespace
}  // namespace pattn

using namespace pattn;

extern "C" size_t pattn_latent_workspace_bytes(int num_seqs, int num_heads, int latent_size) {
  if (num_seqs < 0 || num_heads <= 0 || latent_size <= 0 || latent_size % 128 != 0 ||
      latent_size > 512)
    return 0;
  return la_layout(num_seqs, latent_size).total;
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
  const LaLayout l = la_layout(a->num_seqs, a->latent_size);
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
  p.cuts = reinterpret_cast<Cut*>(ws + l.cuts);
  p.prefix = reinterpret_cast<double*>(ws + l.prefix);
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
  const int tiles = (a->num_heads + R - 1) / R;  // row tiles of a token
  p.lanes = a->max_query_len <= 1 && tiles > 1 && tiles <= 8 ? tiles : 1;
  p.max_shares = std::max(1, l.grid / p.lanes);
  // a copy is a run of rows of one block: 64, 32 or 16
  p.box = a->block_size % 64 == 0 ? 64 : a->block_size % 32 == 0 ? 32 : 16;
  const int dim = a->latent_size + a->rope_size;
  CUtensorMap qmap, cmap;
  if (!encode_rows_map(&qmap, a->q, p.half, dim, 1, a->num_tokens * a->num_heads, dim, dim, R) ||
      !encode_rows_map(&cmap, a->kv_cache, p.half, dim, 1, a->num_blocks * a->block_size, dim, dim,
                       p.box))
    return PATTN_ERR_CUDA;
  const int grid = p.max_shares * p.lanes;
  cudaStream_t st = static_cast<cudaStream_t>(a->stream);
  const cudaError_t e = R == 16   ? launch_latent_rows<16>(p, qmap, cmap, grid, st)
                        : R == 32 ? launch_latent_rows<32>(p, qmap, cmap, grid, st)
                                  : launch_latent_rows<64>(p, qmap, cmap, grid, st);
  return e == cudaSuccess ? PATTN_OK : PATTN_ERR_CUDA;
}
