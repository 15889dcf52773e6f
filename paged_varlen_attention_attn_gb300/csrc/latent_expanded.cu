// latent_expanded.cu -- attention over keys and values that were projected up from
// a shared latent vector, one pair per head, with a rotary key that all heads share
// (sm_103a).
//
//   out_i = sum_k p_ik v_k,   p_i = softmax_k scale (qn_i . kn_k + qr_i . kr_k)
// over the visible keys k of the row's request: q = [qn (dn) | qr (dr)] and v (dv =
// dn) per head, kr (dr) shared.  Rows are contiguous and ragged: request r has q
// rows [qsl[r], qsl[r + 1]) and keys [ksl[r], ksl[r + 1]); row i sits at position
// keys - queries + i.
//
// Bound by the tensor cores: 2 (dn + dr + dv) flops per pair and head, and each
// key tile is read once per 256 rows.  A persistent CTA owns two 128-row sub-tiles of
// one head and walks their key tiles; S = Q K^T (dn + dr deep) and O += P V are
// tcgen05 MMAs, P stays in TMEM, the softmax is online with a lazy reference max.
//
// Shared memory decides the shape.  Q takes (dn + 64) x 256 x 2 bytes, 96 KB at dn =
// 128, and with tiles of 128 keys (48 KB of K, 32 KB of V) the two sub-tiles taking
// turns on the tensor core, as in the paged prefill kernel of this library, a tile has
// to stay while both use it and too little is left for the copies behind it: 1990 us
// for 8 prompts of 1024 to 8192, 32 heads, whatever the rings were cut into.  So
// tiles are 64 keys, each sub-tile has two score buffers in TMEM (4 x 64 columns beside
// the 2 x dv of O), and both sub-tiles' MMAs on a tile follow each other at once: S_A,
// S_B of tile j + 1, then P V_A, P V_B of tile j, from a warp each.  K and V then have
// three stages, and the softmax of a tile runs under the MMAs of its neighbours: 1780
// to 1810 us, 1.25 PFLOP/s.  The price is S at N 64, which reads operands for 48 cycles
// an MMA against 32 of the tensor core, and bounds it now.  (4 chunks of 2048 behind
// 6144, 16 heads: 469 to 477 us, 1.27 PFLOP/s; 6 short requests 7.7 us on the GPU.  Heads
// of 64, rotary 64, the same prompts: 1175 us, 1.15 PFLOP/s.)
//
// P is rounded to the operands' type, as the tensor core takes it; its sum is not.  (bf16:
// 2.1e-3 from the result in 64 bits in root mean square, relative, where the rounding of
// the result alone is 1.6e-3; f16 2.9e-4 and 2.1e-4.)
//
// Rotary parts shorter than 64 are widened with zeros by TMA (a box that reaches
// past the row), so S is always a whole number of 64-element column blocks.
//
// Sixteen warps: 0-3 and 4-7 softmax and epilogue of the two sub-tiles, 8 TMA of Q
// and K, 9 TMA of V, 10 and 11 the MMAs of S of each sub-tile, 12 and 13 those of P V
// (14 and 15 leave at once).
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstddef>

#include "../../include/pattn.h"
#include "common.cuh"
#include "internal.h"

namespace pattn {
namespace {

constexpr int EX_THREADS = 512;
constexpr int EX_SOFTMAX_REGS = 184, EX_OTHER_REGS = 72;  // setmaxnreg split
constexpr int EX_REGS_TOTAL = 2 * 128 * (EX_SOFTMAX_REGS + EX_OTHER_REGS);
constexpr int EX_ROWS = 256;  // query rows of an item
constexpr int EX_RING = 4;    // item ring
constexpr int EX_FEW = 128;   // items that a CTA lists itself
constexpr int EX_KEYS = 64;   // keys of a tile
constexpr float EX_RESCALE_LOG2 = 8.f;
constexpr float EX_SUM_LIMIT = 256.f;  // 2^EX_RESCALE_LOG2
constexpr unsigned FULL = 0xffffffffu;

struct ExHeader {
  unsigned status;      // (see STATUS_WORDS_SHIFT)
  int tiles;            // written by the plan kernel
  unsigned next_item;   // zeroed by the plan kernel
  int pad[61];
};
static_assert(sizeof(ExHeader) == 256 && offsetof(ExHeader, status) == offsetof(WsHeader, status),
              "the status word is where pattn_read_device_status looks for it");

struct ExProblem {
  const int* qsl;
  const int* ksl;
  void* out;
  ExHeader* hdr;
  unsigned* words;  // behind the header: the CTAs' own status, where few
  int2* tiles;
  int max_tiles;
  int few;  // an item a CTA at most: the CTAs list the items themselves
  int B, T, K, H, causal;
  float sl2;
  int test_skip;  // wait-test build only
};

// NB: 64-element column blocks of the part without rotation (dn = dv = 64 NB).
template <int NB>
struct ExCfg {
  static constexpr int DV = 64 * NB;
  static constexpr int KB = NB + 1;  // column blocks of q and k
  static constexpr int QBLK = BLOCK_M * 128;
  static constexpr int QTILE = KB * QBLK;
  static constexpr int BLK = EX_KEYS * 128;
  static constexpr int KTILE = KB * BLK;
  static constexpr int VTILE = NB * BLK;
  static constexpr int ST = NB == 2 ? 3 : 4;  // stages of K and of V
  static constexpr int K_OFF = 2 * QTILE;
  static constexpr int V_OFF = K_OFF + ST * KTILE;
  static constexpr int BAR_OFF = V_OFF + ST * VTILE;
  static constexpr int SMEM = BAR_OFF + 512 + 1024;
  static_assert(SMEM <= 232448 && SMEM > 118784, "one CTA fills an SM");
  // TMEM columns of sub-tile X's score buffer b (P takes its lower half) and output
  __device__ static constexpr unsigned s_col(int X, int b) { return X * 128u + b * EX_KEYS; }
  __device__ static constexpr unsigned o_col(int X) { return X ? 384u : 256u; }
};

struct ExBars {
  uint64_t q_full[2], q_empty, k_full[4], k_empty[4], v_full[4], v_empty[4];
  // by sub-tile and score buffer (a phase of one waits for the last one's reader):
  // scores there, weights there, P V of the weights done
  uint64_t s_full[2][2], p_full[2][2], pv_done[2][2];
  uint64_t v_clean[4];  // a V stage's rows behind the request's keys are zero
  uint64_t drain[4];
  uint64_t ring_full[EX_RING], ring_empty[EX_RING];
  int ring[EX_RING];
  unsigned status;  // of this CTA
  unsigned tmem_base;
  int abort_flag;
};
static_assert(sizeof(ExBars) <= 512, "the barriers fit the space kept for them");

// ------------------------------------------------------------------- plan

__device__ __forceinline__ bool ex_request(const ExProblem& p, int r, int& t0, int& q, int& k0,
                                           int& s) {
  t0 = p.qsl[r];
  q = p.qsl[r + 1] - t0;
  k0 = p.ksl[r];
  s = p.ksl[r + 1] - k0;
  return q >= 0 && s >= 0 && t0 >= 0 && k0 >= 0 && q <= p.T - t0 && s <= p.K - k0 &&
         (!p.causal || q <= s);
}

// The rows of a bad request that lie inside out.
__device__ __forceinline__ void ex_clip(const ExProblem& p, int& t0, int& q) {
  const int64_t end = static_cast<int64_t>(t0) + q;
  t0 = min(max(t0, 0), p.T);
  q = static_cast<int>(max(static_cast<int64_t>(0), min(end, static_cast<int64_t>(p.T)) - t0));
}

__device__ __forceinline__ int ex_tiles_seen(const ExProblem& p, int q, int s, int row_end) {
  const int hi = p.causal ? min(s, s - q + row_end) : s;
  return (hi + EX_KEYS - 1) / EX_KEYS;
}

constexpr int EX_BUCKETS = 2048;
constexpr int EX_PLAN_THREADS = 512;

// The items (request, 256 rows) by their number of key tiles, largest first: a
// counting sort in one CTA.
__global__ void __launch_bounds__(EX_PLAN_THREADS)
    expanded_plan_kernel(const __grid_constant__ ExProblem p) {
  __shared__ int hist[EX_BUCKETS];
  __shared__ int warp_sums[EX_PLAN_THREADS / 32];
  __shared__ unsigned bad;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  grid_dep_trigger();
  grid_dep_wait();
  for (int b = tid; b < EX_BUCKETS; b += EX_PLAN_THREADS) hist[b] = 0;
  if (tid == 0) {
    bad = 0u;
    p.hdr->next_item = 0u;
  }
  __syncthreads();
  // pass 0 counts, pass 1 places; a warp takes a request, its lanes the tiles
  for (int pass = 0; pass < 2; ++pass) {
    for (int r = wid; r < p.B; r += EX_PLAN_THREADS / 32) {
      int t0, q, k0, s;
      const bool ok = ex_request(p, r, t0, q, k0, s);
      if (!ok) {
        // its rows inside out become items without keys, which write zeros
        if (pass == 0 && lane == 0) bad = PATTN_DEV_BAD_METADATA;
        ex_clip(p, t0, q);
        s = 0;
      }
      for (int qt = lane; qt * EX_ROWS < q; qt += 32) {
        const int c = ok ? min(ex_tiles_seen(p, q, s, min(q, (qt + 1) * EX_ROWS)), EX_BUCKETS - 1) : 0;
        const int at = atomicAdd(&hist[c], 1);
        if (pass == 1 && at < p.max_tiles) p.tiles[at] = make_int2(r, ok ? qt : -1 - qt);
      }
    }
    __syncthreads();
    if (pass == 1) break;
    // bucket b's items start at the number of items in larger buckets
    constexpr int PER = EX_BUCKETS / EX_PLAN_THREADS;
    int v[PER], sum = 0;
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      v[e] = hist[EX_BUCKETS - 1 - (tid * PER + e)];
      sum += v[e];
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(FULL, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) warp_sums[wid] = incl;
    __syncthreads();
    int run = incl - sum;
    for (int w = 0; w < wid; ++w) run += warp_sums[w];
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      hist[EX_BUCKETS - 1 - (tid * PER + e)] = run;
      run += v[e];
    }
    if (tid == EX_PLAN_THREADS - 1) {
      p.hdr->tiles = min(run, p.max_tiles);
      if (run > p.max_tiles) bad = PATTN_DEV_BAD_METADATA;
    }
    __syncthreads();
  }
  if (tid == 0) p.hdr->status = bad;
}

// ------------------------------------------------------------------ attention

// A work item: 256 rows of one head of one request.
struct ExItem {
  int h, i0, t0, q, k0, s;
  bool live;
};

__device__ __forceinline__ ExItem ex_load_item(const ExProblem& p, const int2* tiles, int item,
                                               int n_items) {
  ExItem it;
  it.live = item < n_items;
  it.h = it.i0 = it.t0 = it.q = it.k0 = it.s = 0;
  if (it.live) {
    it.h = item % p.H;
    const int2 tl = tiles[item / p.H];
    it.t0 = p.qsl[tl.x];
    it.q = p.qsl[tl.x + 1] - it.t0;
    if (tl.y >= 0) {
      it.i0 = tl.y * EX_ROWS;
      it.k0 = p.ksl[tl.x];
      it.s = p.ksl[tl.x + 1] - it.k0;
    } else {
      it.i0 = (-1 - tl.y) * EX_ROWS;
      ex_clip(p, it.t0, it.q);
    }
  }
  return it;
}

// Sub-tile X of an item and its number of key tiles.
struct ExSub {
  int i0, n;
  bool valid;
};
__device__ __forceinline__ ExSub ex_sub(const ExProblem& p, const ExItem& it, int X) {
  ExSub u;
  u.i0 = it.i0 + X * BLOCK_M;
  u.valid = it.live && u.i0 < it.q;
  u.n = u.valid ? max(0, ex_tiles_seen(p, it.q, it.s, min(it.q, u.i0 + BLOCK_M))) : 0;
  return u;
}

// The weights 2^(x sl2 - ref) of 32 scores, packed in pairs as P; returns their sum.
template <bool HALF>
__device__ __forceinline__ float ex_weights(const float (&x)[32], float sl2, float ref,
                                            unsigned (&pk)[16]) {
  float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
  for (int e = 0; e < 32; e += 4) {
    float a0 = x[e], a1 = x[e + 1], a2 = x[e + 2], a3 = x[e + 3];
    ffma2(a0, a1, sl2, -ref);
    ffma2(a2, a3, sl2, -ref);
    a0 = fast_exp2(a0);
    a1 = fast_exp2(a1);
    a2 = fast_exp2(a2);
    a3 = fast_exp2(a3);
    fadd2(s0, s1, a0, a1);
    fadd2(s2, s3, a2, a3);
    pk[e / 2] = pack2<HALF>(a0, a1);
    pk[e / 2 + 1] = pack2<HALF>(a2, a3);
  }
  return (s0 + s1) + (s2 + s3);
}

// Every role walks the same items and keeps its ring positions and phases as
// running counts across them, so the next item's loads and first scores overlap
// the end of the current one.  Q is reloaded only after the commit behind the
// item's last scores (q_empty); the first P V of the next item, which overwrites
// O, waits for weights that the softmax warps hand over after their epilogue has
// read O.
template <int NB, bool HALF>
__global__ void __launch_bounds__(EX_THREADS, 1)
    expanded_kernel(const __grid_constant__ ExProblem p, const __grid_constant__ CUtensorMap qmap,
                    const __grid_constant__ CUtensorMap kmap,
                    const __grid_constant__ CUtensorMap rmap,
                    const __grid_constant__ CUtensorMap vmap,
                    const __grid_constant__ CUtensorMap qrmap) {
  using C = ExCfg<NB>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  ExBars* bars = reinterpret_cast<ExBars*>(smem + C::BAR_OFF);
  unsigned* status = &bars->status;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->q_full[i], 1);
      mbar_init(&bars->drain[i], 1);
      mbar_init(&bars->drain[2 + i], 1);
      for (int b = 0; b < 2; ++b) {
        mbar_init(&bars->s_full[i][b], 1);
        mbar_init(&bars->p_full[i][b], BLOCK_M);
        mbar_init(&bars->pv_done[i][b], 1);
      }
    }
    for (int i = 0; i < C::ST; ++i) {
      mbar_init(&bars->k_full[i], 1);
      mbar_init(&bars->k_empty[i], 2);  // one arrival of each sub-tile
      mbar_init(&bars->v_full[i], 1);
      mbar_init(&bars->v_empty[i], 2);
      mbar_init(&bars->v_clean[i], 1);
    }
    mbar_init(&bars->q_empty, 2);
    // the item ring: posted by warp 8; taken by warps 9 to 13 and each softmax warp
    for (int i = 0; i < EX_RING; ++i) {
      mbar_init(&bars->ring_full[i], 1);
      mbar_init(&bars->ring_empty[i], 5 + 8);
    }
    bars->abort_flag = 0;
    bars->status = 0u;
    fence_mbar_init();
    tma_prefetch_desc(&qmap);
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&rmap);
    tma_prefetch_desc(&vmap);
    tma_prefetch_desc(&qrmap);
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
  grid_dep_trigger();
  grid_dep_wait();  // the plan kernel's list, or whatever came before
#ifdef PATTN_WAIT_TEST
  // wait-test build: a first CTA that starts late, some 40 ms behind the others
  if (p.test_skip == 5 && blockIdx.x == 0)
    for (int i = 0; i < 40; ++i) __nanosleep(1000000u);
#endif
  const int2* tiles = p.tiles;
  int n_items;
  if (p.few) {
    // An item a CTA: their order does not matter, and a call without the plan kernel
    // is 4 us shorter.  Thread r places the items of request r.
    __shared__ int2 few_tiles[EX_FEW];
    __shared__ int warp_tiles[EX_THREADS / 32];
    const int r = threadIdx.x;
    int t0 = 0, q = 0, k0, s;
    bool fine = true;
    if (r < p.B && !(fine = ex_request(p, r, t0, q, k0, s))) ex_clip(p, t0, q);
    const int mine = (q + EX_ROWS - 1) / EX_ROWS;
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(FULL, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) warp_tiles[warp] = incl;
    const bool bad = __syncthreads_or(!fine);
    int at = incl - mine, total = 0;
    for (int w = 0; w < EX_THREADS / 32; ++w) {
      if (w < warp) at += warp_tiles[w];
      total += warp_tiles[w];
    }
    for (int t = 0; t < mine && at + t < p.max_tiles; ++t)
      few_tiles[at + t] = make_int2(r, fine ? t : -1 - t);
    if (blockIdx.x == 0 && threadIdx.x == 0)
      p.hdr->status = (gridDim.x << STATUS_WORDS_SHIFT) |
                      (bad || total > p.max_tiles ? PATTN_DEV_BAD_METADATA : 0u);
    n_items = min(total, p.max_tiles) * p.H;
    tiles = few_tiles;
    __syncthreads();
  } else {
    n_items = p.hdr->tiles * p.H;
  }

  // The CTA's k-th item: its own block index, then whatever is next in the list,
  // claimed one ahead by warp 8.  An index of n_items or more ends the sequence.
  auto claim = [&](int k) -> int {
    int idx = k == 0  ? static_cast<int>(blockIdx.x)
              : p.few ? n_items
                      : static_cast<int>(gridDim.x + atomicAdd(&p.hdr->next_item, 1u));
    idx = min(idx, n_items);
    const int slot = k % EX_RING;
    if (k >= EX_RING &&
        !mbar_wait(&bars->ring_empty[slot], ((k / EX_RING) - 1) & 1, status, abort_flag))
      return -1;
    bars->ring[slot] = idx;
    mbar_arrive(&bars->ring_full[slot]);
    return idx;
  };
  auto take = [&](int k) -> int {
    const int slot = k % EX_RING;
    if (!mbar_wait(&bars->ring_full[slot], (k / EX_RING) & 1, status, abort_flag)) return -1;
    return *reinterpret_cast<volatile int*>(&bars->ring[slot]);
  };
  auto release = [&](int k) { mbar_arrive(&bars->ring_empty[k % EX_RING]); };

  unsigned char* sQ = smem;
  unsigned char* sK = smem + C::K_OFF;
  unsigned char* sV = smem + C::V_OFF;

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(EX_OTHER_REGS));
    if (warp == 8 && lane == 0) {
      // ------------------------------------------------------------ Q and K
#ifdef PATTN_WAIT_TEST
      // wait-test build: this tile posts no bytes and issues no copy
      const int skip_pos = (p.test_skip == 4 && blockIdx.x == 0) ||
                                   (p.test_skip == 5 && blockIdx.x + 1 == gridDim.x)
                               ? 0
                               : -1;
#else
      constexpr int skip_pos = -1;
#endif
      int jg = 0, n_worked = 0, armed_end = 0, q_arms0 = 0, q_arms1 = 0;
      bool ok = true;
      int idx = claim(0);
      for (int k = 0; idx >= 0; ++k) {
        const ExItem it = ex_load_item(p, tiles, idx, n_items);
        if (!it.live) break;
        idx = claim(k + 1);
        if (idx < 0) {
          ok = false;
          break;
        }
        const ExSub a = ex_sub(p, it, 0), b = ex_sub(p, it, 1);
        const int n = max(a.n, b.n);
        if (n == 0) continue;
        if (n_worked > 0 && !mbar_wait(&bars->q_empty, (n_worked - 1) & 1, status, abort_flag)) {
          ok = false;
          break;
        }
#pragma unroll
        for (int X = 0; X < 2; ++X) {
          const ExSub& u = X ? b : a;
          if (u.n == 0) continue;
          mbar_arrive_expect_tx(&bars->q_full[X], C::QTILE);
          ++(X ? q_arms1 : q_arms0);
          tma_load_4d(sQ + X * C::QTILE, &qmap, &bars->q_full[X], 0, it.t0 + u.i0, 0, it.h);
          tma_load_4d(sQ + X * C::QTILE + NB * C::QBLK, &qrmap, &bars->q_full[X], 0, it.t0 + u.i0,
                      0, it.h);
        }
        for (int j = 0; j < n; ++j, ++jg) {
          const int st = jg % C::ST;
          if (jg >= C::ST &&
              !mbar_wait(&bars->k_empty[st], ((jg / C::ST) - 1) & 1, status, abort_flag)) {
            ok = false;
            break;
          }
          armed_end = jg + 1;
          if (jg == skip_pos) continue;
          mbar_arrive_expect_tx(&bars->k_full[st], C::KTILE);
          const int row = it.k0 + j * EX_KEYS;
          tma_load_4d(sK + st * C::KTILE, &kmap, &bars->k_full[st], 0, row, 0, it.h);
          tma_load_4d(sK + st * C::KTILE + NB * C::BLK, &rmap, &bars->k_full[st], 0, row, 0, 0);
        }
        if (!ok) break;
        ++n_worked;
      }
      // A role gave up on a wait: no copy may still be writing shared memory when
      // the CTA exits.
      if (!ok || idx < 0 || *abort_flag) {
        drain_armed(bars->k_full, C::ST, armed_end, skip_pos, status);
        if (q_arms0 > 0) mbar_wait(&bars->q_full[0], (q_arms0 - 1) & 1, status, nullptr);
        if (q_arms1 > 0) mbar_wait(&bars->q_full[1], (q_arms1 - 1) & 1, status, nullptr);
      }
    } else if (warp == 9 && lane == 0) {
      // ------------------------------------------------------------------ V
      int jg = 0, armed_end = 0;
      bool ok = true;
      for (int k = 0; ok; ++k) {
        const int idx = take(k);
        if (idx < 0) {
          ok = false;
          break;
        }
        release(k);
        const ExItem it = ex_load_item(p, tiles, idx, n_items);
        if (!it.live) break;
        const int n = max(ex_sub(p, it, 0).n, ex_sub(p, it, 1).n);
        for (int j = 0; j < n; ++j, ++jg) {
          const int st = jg % C::ST;
          if (jg >= C::ST &&
              !mbar_wait(&bars->v_empty[st], ((jg / C::ST) - 1) & 1, status, abort_flag)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&bars->v_full[st], C::VTILE);
          armed_end = jg + 1;
          tma_load_4d(sV + st * C::VTILE, &vmap, &bars->v_full[st], 0, it.k0 + j * EX_KEYS, 0, it.h);
        }
      }
      if (!ok || *abort_flag) drain_armed(bars->v_full, C::ST, armed_end, -1, status);
    } else if (warp >= 10 && warp < 14) {
      // ---------------------------------------------------------------- MMAs
      // A warp each for S and for P V of each sub-tile, so that one's waits and commits
      // pass under the others' MMAs.  The whole warp walks, with what the descriptors
      // are made of known to be the same in all lanes, and the elected lane issues.
      const bool scores = warp < 12;
      const int X = warp & 1;
      const unsigned lead = elect_one();
      constexpr unsigned idesc_s = make_idesc_f16(BLOCK_M, EX_KEYS, !HALF, false);
      constexpr unsigned idesc_pv = make_idesc_f16(BLOCK_M, C::DV, !HALF, true);
      const unsigned t_base = __reduce_max_sync(FULL, tmem);
      const uint64_t q_d = smem_desc_sw128(smem_u32(sQ + X * C::QTILE), 16, 1024);
      const uint64_t k_d = smem_desc_sw128(smem_u32(sK), 16, 1024);
      const uint64_t v_d = smem_desc_sw128(smem_u32(sV), C::BLK, 1024);
      int jg = 0;     // key tiles of the items so far (ring position)
      int cnt = 0;    // of this sub-tile (its score buffer and phase)
      int q_tot = 0;  // its Q tiles
      unsigned clean = 0u;  // sub-tile 0: the phase of each V stage's next clearing, a bit each
      bool ok = true;
      for (int k = 0; ok; ++k) {
        const int idx = take(k);
        if (!__all_sync(FULL, idx >= 0)) break;
        if (lane == 0) release(k);
        const ExItem it = ex_load_item(p, tiles, idx, n_items);
        if (!__any_sync(FULL, it.live)) break;
        const int mine = static_cast<int>(
            __reduce_max_sync(FULL, static_cast<unsigned>(ex_sub(p, it, X).n)));
        const int other = static_cast<int>(
            __reduce_max_sync(FULL, static_cast<unsigned>(ex_sub(p, it, 1 - X).n)));
        const int n = max(mine, other);
        const bool two = other > 0;
        if (n == 0) continue;
        if (scores && mine > 0) {
          if (!__all_sync(FULL, mbar_wait(&bars->q_full[X], q_tot & 1, status, abort_flag))) break;
          ++q_tot;
        }
        for (int j = 0; j < n; ++j, ++jg) {
          const int st = jg % C::ST, b = cnt & 1;
          const bool active = j < mine;
          uint64_t* empty = scores ? &bars->k_empty[st] : &bars->v_empty[st];
          bool there = mbar_wait(scores ? &bars->k_full[st] : &bars->v_full[st], (jg / C::ST) & 1,
                                 status, abort_flag);
          if (active && scores && cnt >= 2)  // the buffer's last weights are used
            there = there &&
                    mbar_wait(&bars->pv_done[X][b], ((cnt >> 1) - 1) & 1, status, abort_flag);
          if (active && !scores)
            there = there && mbar_wait(&bars->p_full[X][b], (cnt >> 1) & 1, status, abort_flag);
          if (!__all_sync(FULL, there)) {
            ok = false;
            break;
          }
          if (!active) {  // nothing for this sub-tile (released only now that it is full:
                          // the barrier counts one arrival of each sub-tile per phase)
            if (lead) mbar_arrive(empty);
            if (it.s - j * EX_KEYS < EX_KEYS) clean ^= 1u << st;
            continue;
          }
          tc_fence_after();
          const unsigned s_t = t_base + X * 128u + b * EX_KEYS;
          if (scores) {
            const uint64_t kb = k_d + ((st * C::KTILE) >> 4);
#pragma unroll
            for (int kk = 0; kk < 4 * C::KB; ++kk)
              tc_mma_ss_if(lead, s_t, q_d + (((kk >> 2) * C::QBLK + (kk & 3) * 32) >> 4),
                           kb + (((kk >> 2) * C::BLK + (kk & 3) * 32) >> 4), idesc_s,
                           kk > 0 ? 1u : 0u);
            if (lead) tc_commit(&bars->s_full[X][b]);
          } else {
            // V rows at or past the request's keys become zero: they may hold anything,
            // and 0 * NaN is NaN.  They are in the item's last tile, where sub-tile 1, if
            // it has rows, is active: its warp clears them, and sub-tile 0's waits for it.
            const int rows = it.s - j * EX_KEYS;
            if (rows < EX_KEYS) {
              if (X == 0 && two) {
                if (!__all_sync(FULL, mbar_wait(&bars->v_clean[st], (clean >> st) & 1u, status,
                                                abort_flag))) {
                  ok = false;
                  break;
                }
                clean ^= 1u << st;
              } else {
                for (int e = lane; e < (EX_KEYS - rows) * 8 * NB; e += 32) {
                  const int r = rows + e / (8 * NB), x = e % (8 * NB);
                  *reinterpret_cast<uint4*>(sV + st * C::VTILE + (x >> 3) * C::BLK + r * 128 +
                                            (x & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (X == 1 && lane == 0) mbar_arrive(&bars->v_clean[st]);
              }
            }
            const uint64_t vb = v_d + ((st * C::VTILE) >> 4);
#pragma unroll
            for (int kk = 0; kk < EX_KEYS / 16; ++kk)
              tc_mma_ts_if(lead, t_base + C::o_col(0) + X * 128u, s_t + kk * 8,
                           vb + ((kk * 2048) >> 4), idesc_pv, (j > 0 || kk > 0) ? 1u : 0u);
            if (lead) tc_commit(&bars->pv_done[X][b]);
          }
          if (lead) tc_commit(empty);
          ++cnt;
        }
        if (ok && scores && lead) tc_commit(&bars->q_empty);
      }
      // no MMA may still be running when TMEM is released
      if (lead) {
        tc_commit(&bars->drain[warp - 10]);
        mbar_wait(&bars->drain[warp - 10], 0, status, nullptr);
      }
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(EX_SOFTMAX_REGS));
    // ------------------------------------------------------------ softmax
    const int X = warp >> 2, row = threadIdx.x & 127;
    const unsigned lane_base = tmem + (static_cast<unsigned>((warp & 3) * 32) << 16);
    const unsigned o_t = lane_base + C::o_col(X);
    const float sl2 = p.sl2;
    int cnt = 0;  // key tiles of this sub-tile so far (score buffer and phase)
    bool ok = true;
    for (int k = 0;; ++k) {
      const int idx = take(k);
      if (!__all_sync(FULL, idx >= 0)) break;
      if (lane == 0) release(k);
      const ExItem it = ex_load_item(p, tiles, idx, n_items);
      if (!it.live) break;
      const ExSub u = ex_sub(p, it, X);
      const int i = u.i0 + row, s = it.s;
      const bool row_ok = i < it.q;
      // row i sees keys below kmax; a tile past `edge` needs the mask
      const int kmax = p.causal ? min(s, s - it.q + i + 1) : s;
      const int edge = min(s, p.causal ? s - it.q + u.i0 + 1 : s) - EX_KEYS;
      float m_run = -INFINITY, l_run = 0.f;
      for (int j = 0; j < u.n; ++j, ++cnt) {
        const int b = cnt & 1;
        if (!__all_sync(FULL, mbar_wait(&bars->s_full[X][b], (cnt >> 1) & 1, status, abort_flag))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const unsigned s_t = lane_base + C::s_col(X, b);
        const int key0 = j * EX_KEYS, lim = kmax - key0;
        const bool masked = key0 > edge;
        // Common case: the reference stays; the weights against it are computed in
        // registers, and if any exceeded 2^EX_RESCALE_LOG2 their sum did too and
        // the tile goes down the path below, which takes the row max.
        bool slow = m_run == -INFINITY;
        float ps = 0.f;
        if (!__any_sync(FULL, slow)) {
          float sv[EX_KEYS];
#pragma unroll
          for (int g = 0; g < EX_KEYS / 32; ++g)
            tc_ld32(s_t + g * 32, *reinterpret_cast<float(*)[32]>(&sv[g * 32]));
          tc_wait_ld();
          if (masked) {
#pragma unroll
            for (int q = 0; q < EX_KEYS; ++q) sv[q] = q < lim ? sv[q] : -INFINITY;
          }
          unsigned pk[EX_KEYS / 2];
#pragma unroll
          for (int g = 0; g < EX_KEYS / 32; ++g)
            ps += ex_weights<HALF>(*reinterpret_cast<const float(*)[32]>(&sv[g * 32]), sl2, m_run,
                                   *reinterpret_cast<unsigned(*)[16]>(&pk[g * 16]));
          slow = !(ps <= EX_SUM_LIMIT);
          if (!__any_sync(FULL, slow)) {
#pragma unroll
            for (int g = 0; g < EX_KEYS / 32; ++g)
              tc_st16u(s_t + g * 16, *reinterpret_cast<const unsigned(*)[16]>(&pk[g * 16]));
          }
        }
        if (__any_sync(FULL, slow)) {
          float sv[EX_KEYS];  // the scores again: nothing was stored over them
#pragma unroll
          for (int g = 0; g < EX_KEYS / 32; ++g)
            tc_ld32(s_t + g * 32, *reinterpret_cast<float(*)[32]>(&sv[g * 32]));
          tc_wait_ld();
          if (masked) {
#pragma unroll
            for (int q = 0; q < EX_KEYS; ++q) sv[q] = q < lim ? sv[q] : -INFINITY;
          }
          float m4[4] = {sv[0], sv[1], sv[2], sv[3]};
#pragma unroll
          for (int q = 4; q < EX_KEYS - 4; q += 8) {
            m4[0] = max3(m4[0], sv[q + 0], sv[q + 1]);
            m4[1] = max3(m4[1], sv[q + 2], sv[q + 3]);
            m4[2] = max3(m4[2], sv[q + 4], sv[q + 5]);
            m4[3] = max3(m4[3], sv[q + 6], sv[q + 7]);
          }
          m4[0] = max3(m4[0], sv[EX_KEYS - 4], sv[EX_KEYS - 3]);
          m4[1] = max3(m4[1], sv[EX_KEYS - 2], sv[EX_KEYS - 1]);
          const float mx = max3(fmaxf(m4[0], m4[1]), m4[2], m4[3]);
          const float mx_s = mx == -INFINITY ? -INFINITY : mx * sl2;
          // the reference moves only where a row max grows by more than
          // 2^EX_RESCALE_LOG2 or a row's weights summed above it
          const bool grow = mx_s > m_run + (slow ? 0.f : EX_RESCALE_LOG2);
          const bool need_o = grow && m_run != -INFINITY;
          float alpha = 1.f;
          if (grow) {
            alpha = m_run == -INFINITY ? 0.f : fast_exp2(m_run - mx_s);
            l_run *= alpha;
            m_run = mx_s;
          }
          const float ref = m_run == -INFINITY ? 0.f : m_run;
          ps = 0.f;
#pragma unroll
          for (int g = 0; g < EX_KEYS / 32; ++g) {
            unsigned pk[16];
            ps += ex_weights<HALF>(*reinterpret_cast<const float(*)[32]>(&sv[g * 32]), sl2, ref, pk);
            tc_st16u(s_t + g * 16, pk);
          }
          // O is rescaled last, once the score registers are free and P V of the
          // previous tile is in it.
          if (__any_sync(FULL, need_o)) {
            if (!__all_sync(FULL, mbar_wait(&bars->pv_done[X][b ^ 1], ((cnt - 1) >> 1) & 1, status,
                                            abort_flag))) {
              ok = false;
              break;
            }
            tc_fence_after();
            const float a = need_o ? alpha : 1.f;
#pragma unroll
            for (int q = 0; q < C::DV / 32; ++q) {
              float ov[32];
              tc_ld32(o_t + q * 32, ov);
              tc_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) ov[e] *= a;
              tc_st32(o_t + q * 32, ov);
            }
          }
        }
        l_run += ps;
        tc_wait_st();
        tc_fence_before();
        mbar_arrive(&bars->p_full[X][b]);
      }
      if (!ok) break;

      // --------------------------------------------------------- epilogue
      if (!u.valid) continue;
      if (u.n > 0) {
        if (!__all_sync(FULL, mbar_wait(&bars->pv_done[X][(cnt - 1) & 1], ((cnt - 1) >> 1) & 1,
                                        status, abort_flag)))
          break;
        tc_fence_after();
      }
      const float inv = l_run > 0.f ? 1.f / l_run : l_run == 0.f ? 0.f : NAN;
      uint16_t* orow = static_cast<uint16_t*>(p.out) +
                       (static_cast<int64_t>(it.t0 + i) * p.H + it.h) * C::DV;
#pragma unroll
      for (int q = 0; q < C::DV / 32; ++q) {
        float ov[32];
        if (u.n > 0) {
          tc_ld32(o_t + q * 32, ov);
          tc_wait_ld();
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) ov[e] = 0.f;
        }
        if (row_ok) {
          unsigned w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) w[e] = pack2<HALF>(ov[2 * e] * inv, ov[2 * e + 1] * inv);
#pragma unroll
          for (int e = 0; e < 16; e += 4)
            *reinterpret_cast<uint4*>(orow + q * 32 + e * 2) =
                make_uint4(w[e], w[e + 1], w[e + 2], w[e + 3]);
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0) {
    // (the plan kernel has cleared the call's word; in a call without one, the first CTA
    // may do so after this one has ended)
    if (p.few) p.words[blockIdx.x] = bars->status;
    else if (bars->status) flag_status(&p.hdr->status, bars->status);
  }
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

struct ExLayout {
  int max_tiles;
  size_t tiles_off, total;
};

ExLayout ex_layout(int B, int T) {
  ExLayout l;
  l.max_tiles = T / EX_ROWS + B;  // a request's last item may be short
  l.tiles_off = sizeof(ExHeader) + MAX_STATUS_WORDS * sizeof(unsigned);
  l.total = l.tiles_off + (static_cast<size_t>(l.max_tiles) * sizeof(int2) + 255) / 256 * 256;
  return l;
}

template <int NB, bool HALF>
cudaError_t launch_expanded(const ExProblem& p, const CUtensorMap (&m)[5], cudaStream_t st) {
  using C = ExCfg<NB>;
  auto kern = expanded_kernel<NB, HALF>;
  static std::atomic<unsigned long long> ready{0};  // devices whose limit is set
  cudaError_t e = cudaSuccess;
  if (!p.few) {
    e = launch_dependent(expanded_plan_kernel, dim3(1), EX_PLAN_THREADS, 0, st, p);
    if (e != cudaSuccess) return e;
  }
  const dim3 grid(static_cast<unsigned>(
      std::min<long long>(static_cast<long long>(p.max_tiles) * p.H, current_sms())));
  e = cudaErrorInvalidValue;
  for (int again = 0; again < 2 && e == cudaErrorInvalidValue; ++again) {
    // (with the limit: the register split must fit in what the CTA is launched with)
    e = allow_shared_memory(reinterpret_cast<const void*>(kern), C::SMEM, ready, again, EX_THREADS,
                            EX_REGS_TOTAL);
    if (e != cudaSuccess) return e;
    e = launch_dependent(kern, grid, EX_THREADS, C::SMEM, st, p, m[0], m[1], m[2], m[3], m[4]);
    if (e == cudaErrorInvalidValue) cudaGetLastError();
  }
  return e;
}

}  // namespace
}  // namespace pattn

using namespace pattn;

extern "C" size_t pattn_latent_expanded_workspace_bytes(int num_seqs, int num_tokens) {
  return num_seqs < 0 || num_tokens < 0 ? 0 : ex_layout(num_seqs, num_tokens).total;
}

extern "C" pattn_status_t pattn_latent_expanded_fwd(const pattn_latent_expanded_t* a) {
  if (!a || a->struct_size < sizeof(pattn_latent_expanded_t)) return PATTN_ERR_INVALID_ARGUMENT;
  if (!a->q || !a->k_nope || !a->k_rope || !a->value || !a->out || !a->query_start_loc ||
      !a->key_start_loc || !a->workspace)
    return PATTN_ERR_INVALID_ARGUMENT;
  if (a->num_seqs < 0 || a->num_tokens < 0 || a->num_keys < 0 || a->num_heads <= 0 ||
      a->nope_size <= 0 || a->rope_size <= 0 || a->value_size <= 0)
    return PATTN_ERR_INVALID_ARGUMENT;
  if (!(a->scale >= 0.f) || std::isinf(a->scale) || (a->causal != 0 && a->causal != 1))
    return PATTN_ERR_INVALID_ARGUMENT;
  if ((a->nope_size != 64 && a->nope_size != 128) || a->value_size != a->nope_size ||
      a->rope_size % 16 != 0 || a->rope_size > 64)
    return PATTN_ERR_UNSUPPORTED;
  if (a->kv_dtype != PATTN_KV_BF16 && a->kv_dtype != PATTN_KV_F16) return PATTN_ERR_UNSUPPORTED;
  for (const void* x : {a->q, a->k_nope, a->k_rope, a->value, static_cast<const void*>(a->out)})
    if (reinterpret_cast<uintptr_t>(x) & 15) return PATTN_ERR_INVALID_ARGUMENT;
  if (reinterpret_cast<uintptr_t>(a->workspace) & 255) return PATTN_ERR_INVALID_ARGUMENT;
  for (const long long s : {a->q_stride, a->q_head_stride, a->k_stride, a->k_head_stride,
                            a->k_rope_stride, a->v_stride, a->v_head_stride})
    if (s <= 0 || s % 8 != 0 || s > (1LL << 38)) return PATTN_ERR_INVALID_ARGUMENT;
  const ExLayout l = ex_layout(a->num_seqs, a->num_tokens);
  if (a->workspace_bytes < l.total) return PATTN_ERR_WORKSPACE_TOO_SMALL;
  if (static_cast<long long>(l.max_tiles) * a->num_heads > (1 << 30)) return PATTN_ERR_UNSUPPORTED;
  if (a->num_seqs == 0 || a->num_tokens == 0) return PATTN_OK;
  ExProblem p = {};
  p.qsl = a->query_start_loc;
  p.ksl = a->key_start_loc;
  p.out = a->out;
  p.hdr = static_cast<ExHeader*>(a->workspace);
  p.words = reinterpret_cast<unsigned*>(p.hdr + 1);
  p.tiles = reinterpret_cast<int2*>(static_cast<unsigned char*>(a->workspace) + l.tiles_off);
  p.max_tiles = l.max_tiles;
  p.B = a->num_seqs;
  p.T = a->num_tokens;
  p.K = a->num_keys;
  p.H = a->num_heads;
  p.causal = a->causal;
  p.few = l.max_tiles <= EX_FEW &&
          static_cast<long long>(l.max_tiles) * a->num_heads <=
              std::min(current_sms(), MAX_STATUS_WORDS);
#ifdef PATTN_WAIT_TEST
  p.test_skip = test_wait_skip();
#endif
  // strictly positive, so that a masked score (-inf) always maps to weight 0; at
  // scale 0 the weights are 1 exactly
  p.sl2 = fmaxf(a->scale * LOG2E, 1e-30f);
  const bool half = a->kv_dtype == PATTN_KV_F16;
  const int H = a->num_heads, keys = std::max(1, a->num_keys);
  const int dn = a->nope_size, dr = a->rope_size;
  const uint16_t* q_rope = static_cast<const uint16_t*>(a->q) + dn;
  CUtensorMap m[5];
  if (!encode_rows_map(&m[0], a->q, half, dn, H, a->num_tokens, a->q_head_stride, a->q_stride,
                       BLOCK_M) ||
      !encode_rows_map(&m[1], a->k_nope, half, dn, H, keys, a->k_head_stride, a->k_stride, EX_KEYS) ||
      !encode_rows_map(&m[2], a->k_rope, half, dr, 1, keys, a->k_rope_stride, a->k_rope_stride,
                       EX_KEYS) ||
      !encode_rows_map(&m[3], a->value, half, dn, H, keys, a->v_head_stride, a->v_stride, EX_KEYS) ||
      !encode_rows_map(&m[4], q_rope, half, dr, H, a->num_tokens, a->q_head_stride, a->q_stride,
                       BLOCK_M))
    return PATTN_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(a->stream);
  const cudaError_t e = a->nope_size == 128
                            ? (half ? launch_expanded<2, true>(p, m, st) : launch_expanded<2, false>(p, m, st))
                            : (half ? launch_expanded<1, true>(p, m, st) : launch_expanded<1, false>(p, m, st));
  return e == cudaSuccess ? PATTN_OK : PATTN_ERR_CUDA;
}
