// latent_cache.cu -- writing and reading back a paged cache of latent rows (sm_103a).
//
// A model with keys and values from one shared latent vector a token caches, per
// token, one row [c (dc) | k (dr)]: the latent c and a rotary key k that all
// heads share.  The cache is [num_blocks][block_size][dc + dr], 16-bit.
//
// The write does, for each token, c <- c * rsqrt(mean(c^2) + eps) * w if a norm's
// weight is given, turns k and the rotary part of every q head by the token's
// position, (a, b) -> (a cos - b sin, b cos + a sin), and stores c and k as the
// token's cache row (and, if asked, as a dense row, the input of the
// up-projection).  fp32 throughout with one rounding at the end.
//
// Both are bound by HBM: every byte is read once and written once.  8384 tokens of 64
// heads with the dense row: 28.3 us a call, 5.97 TB/s; 64 requests of 512 to 4096 keys read
// back: 52.6 us, 6.35 TB/s.  A token or a few hundred keys are a chain of latencies,
// 1.9 and 2.9 us on the GPU.
#include <algorithm>
#include <cmath>

#include "../../include/pattn.h"
#include "common.cuh"
#include "internal.h"

namespace pattn {
namespace {

constexpr int LW_THREADS = 128;
constexpr int LW_STEPS = 4;  // q steps of a warp where there are many tokens

struct WriteParams {
  const uint16_t* q;
  uint16_t* q_out;
  const uint16_t* latent;
  const uint16_t* k_rope;
  const uint16_t* norm;
  uint16_t* cache;
  uint16_t* row_out;
  const float* table;  // [max_pos][dr]: cos, then sin
  const int64_t* positions;
  const int64_t* slots;
  unsigned* status;
  int64_t q_ts, q_hs, qo_ts, qo_hs, c_ts, k_ts, row_ts;  // elements between tokens / heads
  int64_t pool;                                          // slots of the cache
  float eps, inv_dc;
  int T, H, dc, dr, max_pos, adjacent;
  int steps_q;  // steps of 32 / LPR heads of a token
  int units;    // warps of a token: its q steps by the warp's count, and one for its row
};

// The two pieces of a rotary row that one lane holds, turned.  In halves the
// pieces are partners (element e of the first with element e of the second);
// adjacent pairs lie inside each piece.  cs, sn: the lane's eight pairs.
template <bool HALF>
__device__ __forceinline__ void turn_pieces(uint4& wa, uint4& wb, const float (&cs)[8],
                                            const float (&sn)[8], bool adjacent) {
  float x[8], y[8];
  unpack8<HALF>(wa, x);
  unpack8<HALF>(wb, y);
  if (adjacent) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float a = x[2 * e], b = x[2 * e + 1], c = y[2 * e], d = y[2 * e + 1];
      x[2 * e] = a * cs[e] - b * sn[e];
      x[2 * e + 1] = b * cs[e] + a * sn[e];
      y[2 * e] = c * cs[4 + e] - d * sn[4 + e];
      y[2 * e + 1] = d * cs[4 + e] + c * sn[4 + e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float a = x[e], b = y[e];
      x[e] = a * cs[e] - b * sn[e];
      y[e] = b * cs[e] + a * sn[e];
    }
  }
  wa = pack8<HALF>(x);
  wb = pack8<HALF>(y);
}

// A warp serves STEPS steps of 32 / LPR q heads of one token, or the token's
// cache row.  LPR = dr / 16 lanes, rounded up to a power of two, own a rotary
// row, 16 elements each.
template <int LPR, int STEPS, bool HALF>
__global__ void __launch_bounds__(LW_THREADS)
    latent_write_kernel(const __grid_constant__ WriteParams p) {
  constexpr int RPS = 32 / LPR;
  grid_dep_trigger();
  grid_dep_wait();
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * (LW_THREADS / 32) + (threadIdx.x >> 5);
  const int64_t t = unit / p.units;
  if (t >= p.T) return;
  const int u = static_cast<int>(unit - t * p.units);
  const int lane = threadIdx.x & 31;
  const int j = lane % LPR, half = p.dr / 16;
  const bool on = j < half;
  const int c0 = j * 8, c1 = (j + half) * 8;
  const bool row_unit = u == p.units - 1;

  // every load that does not depend on another goes out first
  uint4 wa[STEPS], wb[STEPS];
  uint4 lat[2], lw[2];
  const int h0 = u * STEPS * RPS + lane / LPR;
  const int pieces = p.dc / 8;
  if (!row_unit) {
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const int h = h0 + i * RPS;
      wa[i] = wb[i] = make_uint4(0u, 0u, 0u, 0u);
      if (on && h < p.H) {
        const uint16_t* src = p.q + t * p.q_ts + h * p.q_hs;
        wa[i] = *reinterpret_cast<const uint4*>(src + c0);
        wb[i] = *reinterpret_cast<const uint4*>(src + c1);
      }
    }
  } else {
    wa[0] = wb[0] = make_uint4(0u, 0u, 0u, 0u);
    if (on && lane < LPR) {
      wa[0] = *reinterpret_cast<const uint4*>(p.k_rope + t * p.k_ts + c0);
      wb[0] = *reinterpret_cast<const uint4*>(p.k_rope + t * p.k_ts + c1);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      lat[i] = lw[i] = make_uint4(0u, 0u, 0u, 0u);
      const int c = lane + 32 * i;
      if (c < pieces) {
        lat[i] = *reinterpret_cast<const uint4*>(p.latent + t * p.c_ts + c * 8);
        if (p.norm) lw[i] = *reinterpret_cast<const uint4*>(p.norm + c * 8);
      }
    }
  }
  // a negative position marks padding (nothing of the token is written), one
  // outside the table is reported and the token skipped
  float cs[8], sn[8];
  if (p.positions) {
    const int64_t pos = p.positions[t];
    if (pos < 0 || pos >= p.max_pos) {
      if (pos >= 0 && u == 0 && lane == 0) flag_status(p.status, PATTN_DEV_BAD_METADATA);
      return;
    }
    if (on) {
      const float* r = p.table + pos * p.dr;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int p0 = p.adjacent ? (h ? c1 : c0) / 2 : 8 * j + 4 * h;
        const float4 c = *reinterpret_cast<const float4*>(r + p0);
        const float4 s = *reinterpret_cast<const float4*>(r + p.dr / 2 + p0);
        cs[4 * h] = c.x; cs[4 * h + 1] = c.y; cs[4 * h + 2] = c.z; cs[4 * h + 3] = c.w;
        sn[4 * h] = s.x; sn[4 * h + 1] = s.y; sn[4 * h + 2] = s.z; sn[4 * h + 3] = s.w;
      }
    }
  }
  if (!row_unit) {
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const int h = h0 + i * RPS;
      if (!on || h >= p.H) continue;
      if (p.positions) turn_pieces<HALF>(wa[i], wb[i], cs, sn, p.adjacent);
      uint16_t* d = p.q_out + t * p.qo_ts + h * p.qo_hs;
      *reinterpret_cast<uint4*>(d + c0) = wa[i];
      *reinterpret_cast<uint4*>(d + c1) = wb[i];
    }
    return;
  }
  const int64_t slot = p.slots[t];
  if (p.norm) {
    float x[2][8], ss = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      unpack8<HALF>(lat[i], x[i]);
#pragma unroll
      for (int e = 0; e < 8; ++e) ss += x[i][e] * x[i][e];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float r = rsqrtf(ss * p.inv_dc + p.eps);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float w[8];
      unpack8<HALF>(lw[i], w);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[i][e] *= r * w[e];
      lat[i] = pack8<HALF>(x[i]);
    }
  }
  if (p.positions && on && lane < LPR) turn_pieces<HALF>(wa[0], wb[0], cs, sn, p.adjacent);
  // a negative slot writes no cache row; one past the pool is reported as well
  if (slot >= p.pool && lane == 0) flag_status(p.status, PATTN_DEV_BAD_METADATA);
  uint16_t* dst[2] = {slot >= 0 && slot < p.pool ? p.cache + slot * (p.dc + p.dr) : nullptr,
                      p.row_out ? p.row_out + t * p.row_ts : nullptr};
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (!dst[k]) continue;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (lane + 32 * i < pieces) *reinterpret_cast<uint4*>(dst[k] + (lane + 32 * i) * 8) = lat[i];
    if (on && lane < LPR) {
      *reinterpret_cast<uint4*>(dst[k] + p.dc + c0) = wa[0];
      *reinterpret_cast<uint4*>(dst[k] + p.dc + c1) = wb[0];
    }
  }
}

template <int LPR, int STEPS, bool HALF>
cudaError_t launch_write(WriteParams& p, cudaStream_t st) {
  p.steps_q = (p.H + 32 / LPR - 1) / (32 / LPR);
  p.units = (p.steps_q + STEPS - 1) / STEPS + 1;
  const long long ctas =
      (static_cast<long long>(p.T) * p.units + LW_THREADS / 32 - 1) / (LW_THREADS / 32);
  if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  return launch_dependent(latent_write_kernel<LPR, STEPS, HALF>, dim3(static_cast<unsigned>(ctas)),
                          LW_THREADS, 0, st, p);
}

template <int LPR, bool HALF>
cudaError_t launch_write_lpr(WriteParams& p, cudaStream_t st) {
  // One step a warp until every SM has warps enough to hide the loads' latency, then
  // fewer warps that read the position and the table row again.  (One against four
  // steps, heads of 64: 256 tokens of 128 heads 2.8 and 3.7 us, 512 of 64 2.9 and 3.8;
  // 1024 of 64 4.6 and 4.2, 2048 of 128 12.1 and 8.9.)
  const long long warps = static_cast<long long>(p.T) * ((p.H + 32 / LPR - 1) / (32 / LPR));
  return warps >= 48LL * current_sms() ? launch_write<LPR, LW_STEPS, HALF>(p, st)
                                       : launch_write<LPR, 1, HALF>(p, st);
}

template <bool HALF>
cudaError_t launch_write_type(WriteParams& p, cudaStream_t st) {
  return p.dr <= 16   ? launch_write_lpr<1, HALF>(p, st)
         : p.dr <= 32 ? launch_write_lpr<2, HALF>(p, st)
                      : launch_write_lpr<4, HALF>(p, st);
}

// ---------------------------------------------------------------- read-back

constexpr int GL_THREADS = 128;
constexpr int GL_ROWS = 4;   // rows of a warp
constexpr int GL_BATCH = 9;  // 16-byte pieces a lane has in flight (4 rows of 1152 bytes)

struct ReadParams {
  const uint16_t* cache;
  const int* block_table;
  const int* key_starts;
  const int* osl;
  uint16_t* latent;
  uint16_t* rope;
  unsigned* status;
  int B, rows, mbps, NB, dc, dr, bs;
};

// Output row i belongs to request r with osl[r] <= i < osl[r + 1] and holds key
// key_starts[r] + i - osl[r].  A warp takes GL_ROWS rows: that many lanes find
// their row's request (binary search) and block, then the rows' pieces are
// dealt out to the lanes one after the other.  The kernel alone takes 49.4 us for 145 k
// rows of 1152 bytes, 6.75 TB/s.
__global__ void __launch_bounds__(GL_THREADS)
    gather_latent_kernel(const __grid_constant__ ReadParams p) {
  grid_dep_trigger();
  grid_dep_wait();
  const int64_t first =
      (static_cast<int64_t>(blockIdx.x) * (GL_THREADS / 32) + (threadIdx.x >> 5)) * GL_ROWS;
  if (first >= p.rows) return;
  const int lane = threadIdx.x & 31;
  int64_t slot = -2;  // -2: leave the row, -1: zero it, else the cache slot
  if (lane < GL_ROWS && first + lane < p.rows) {
    const int row = static_cast<int>(first) + lane;
    int lo = 0, hi = p.B;  // the last request that starts at or before the row
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.osl[mid] <= row) lo = mid;
      else hi = mid;
    }
    const int at = p.osl[lo];
    if (row >= at && row < p.osl[lo + 1]) {
      const int64_t key = static_cast<int64_t>(p.key_starts ? p.key_starts[lo] : 0) + row - at;
      int blk = -1;
      if (key >= 0 && key < static_cast<int64_t>(p.mbps) * p.bs)
        blk = p.block_table[static_cast<int64_t>(lo) * p.mbps + key / p.bs];
      if (blk < 0 || blk >= p.NB) {
        flag_status(p.status, PATTN_DEV_BAD_METADATA);
        slot = -1;
      } else {
        slot = static_cast<int64_t>(blk) * p.bs + key % p.bs;
      }
    }
  }
  const int pieces = (p.dc + p.dr) / 8, lat_pieces = p.dc / 8;
  for (int base = 0; base < GL_ROWS * pieces; base += 32 * GL_BATCH) {
    uint4 w[GL_BATCH];
    int64_t from[GL_BATCH];
#pragma unroll
    for (int i = 0; i < GL_BATCH; ++i) {
      const int c = base + 32 * i + lane;
      int r = 0;
#pragma unroll
      for (int k = 1; k < GL_ROWS; ++k) r += c >= k * pieces;
      from[i] = __shfl_sync(0xffffffffu, slot, r);
      if (c >= GL_ROWS * pieces) from[i] = -2;
      w[i] = make_uint4(0u, 0u, 0u, 0u);
      if (from[i] >= 0)
        w[i] = *reinterpret_cast<const uint4*>(p.cache + from[i] * (p.dc + p.dr) +
                                               (c - r * pieces) * 8);
    }
#pragma unroll
    for (int i = 0; i < GL_BATCH; ++i) {
      if (from[i] == -2) continue;
      const int c = base + 32 * i + lane;
      int r = 0;
#pragma unroll
      for (int k = 1; k < GL_ROWS; ++k) r += c >= k * pieces;
      const int e = c - r * pieces;
      uint16_t* dst = e < lat_pieces ? p.latent + (first + r) * p.dc + e * 8
                                     : p.rope + (first + r) * p.dr + (e - lat_pieces) * 8;
      *reinterpret_cast<uint4*>(dst) = w[i];
    }
  }
}

bool misaligned(const void* x) { return (reinterpret_cast<uintptr_t>(x) & 15) != 0; }

}  // namespace

pattn_status_t check_latent_sizes(int latent_size, int rope_size, int block_size, int kv_dtype) {
  if (latent_size <= 0 || rope_size <= 0 || block_size <= 0 || block_size % 16 != 0)
    return PATTN_ERR_INVALID_ARGUMENT;
  if (latent_size % 128 != 0 || latent_size > 512 || rope_size % 16 != 0 || rope_size > 64)
    return PATTN_ERR_UNSUPPORTED;
  if (kv_dtype != PATTN_KV_BF16 && kv_dtype != PATTN_KV_F16) return PATTN_ERR_UNSUPPORTED;
  return PATTN_OK;
}

}  // namespace pattn

using namespace pattn;

extern "C" pattn_status_t pattn_latent_rope_and_cache(const pattn_latent_rope_t* a) {
  if (!a || a->struct_size < sizeof(pattn_latent_rope_t)) return PATTN_ERR_INVALID_ARGUMENT;
  const pattn_status_t v =
      check_latent_sizes(a->latent_size, a->rope_size, a->block_size, a->kv_dtype);
  if (v != PATTN_OK) return v;
  const bool has_q = a->q != nullptr;
  if (has_q != (a->q_out != nullptr) || !a->latent || !a->k_rope || !a->kv_cache ||
      !a->slot_mapping)
    return PATTN_ERR_INVALID_ARGUMENT;
  if (a->num_tokens < 0 || a->num_blocks < 0 || (has_q && a->num_heads <= 0) ||
      (a->interleaved != 0 && a->interleaved != 1))
    return PATTN_ERR_INVALID_ARGUMENT;
  if (a->positions && (!a->cos_sin || misaligned(a->cos_sin) || a->max_position <= 0))
    return PATTN_ERR_INVALID_ARGUMENT;
  if (a->latent_norm && !(a->norm_eps >= 0.f && a->norm_eps < INFINITY))
    return PATTN_ERR_INVALID_ARGUMENT;
  // rows are moved in 16-byte pieces
  if (misaligned(a->q) || misaligned(a->q_out) || misaligned(a->latent) || misaligned(a->k_rope) ||
      misaligned(a->kv_cache) || misaligned(a->row_out) || misaligned(a->latent_norm))
    return PATTN_ERR_INVALID_ARGUMENT;
  const long long strides[] = {has_q ? a->q_stride : 0,     has_q ? a->q_head_stride : 0,
                               has_q ? a->q_out_stride : 0, has_q ? a->q_out_head_stride : 0,
                               a->latent_stride,            a->k_rope_stride,
                               a->row_out ? a->row_out_stride : 0};
  for (const long long s : strides)
    if (s % 8 != 0 || s < 0) return PATTN_ERR_INVALID_ARGUMENT;
  // a written row must not reach into the next one: heads within tokens or tokens
  // within heads
  if (has_q) {
    const long long hs = a->q_out_head_stride, ts = a->q_out_stride, dr = a->rope_size;
    const bool heads_in = hs >= dr && ts >= (a->num_heads - 1) * hs + dr;
    const bool tokens_in = ts >= dr && hs >= (a->num_tokens - 1) * ts + dr;
    if (a->num_heads > 1 && a->num_tokens > 1 && !heads_in && !tokens_in)
      return PATTN_ERR_INVALID_ARGUMENT;
    if (a->num_heads > 1 && hs < dr) return PATTN_ERR_INVALID_ARGUMENT;
    if (a->num_tokens > 1 && ts < dr) return PATTN_ERR_INVALID_ARGUMENT;
  }
  if (a->row_out && a->num_tokens > 1 && a->row_out_stride < a->latent_size + a->rope_size)
    return PATTN_ERR_INVALID_ARGUMENT;
  if (a->num_tokens == 0) return PATTN_OK;
  WriteParams p = {};
  p.q = static_cast<const uint16_t*>(a->q);
  p.q_out = static_cast<uint16_t*>(a->q_out);
  p.latent = static_cast<const uint16_t*>(a->latent);
  p.k_rope = static_cast<const uint16_t*>(a->k_rope);
  p.norm = static_cast<const uint16_t*>(a->latent_norm);
  p.cache = static_cast<uint16_t*>(a->kv_cache);
  p.row_out = static_cast<uint16_t*>(a->row_out);
  p.table = a->cos_sin;
  p.positions = a->positions;
  p.slots = a->slot_mapping;
  p.status = a->device_status;
  p.q_ts = a->q_stride;
  p.q_hs = a->q_head_stride;
  p.qo_ts = a->q_out_stride;
  p.qo_hs = a->q_out_head_stride;
  p.c_ts = a->latent_stride;
  p.k_ts = a->k_rope_stride;
  p.row_ts = a->row_out_stride;
  p.pool = static_cast<int64_t>(a->num_blocks) * a->block_size;
  p.eps = a->norm_eps;
  p.inv_dc = 1.f / static_cast<float>(a->latent_size);
  p.T = a->num_tokens;
  p.H = has_q ? a->num_heads : 0;
  p.dc = a->latent_size;
  p.dr = a->rope_size;
  p.max_pos = a->max_position;
  p.adjacent = a->interleaved;
  cudaStream_t st = static_cast<cudaStream_t>(a->stream);
  const cudaError_t e = a->kv_dtype == PATTN_KV_F16 ? launch_write_type<true>(p, st)
                                                    : launch_write_type<false>(p, st);
  return e == cudaSuccess ? PATTN_OK : PATTN_ERR_CUDA;
}

extern "C" pattn_status_t pattn_gather_latent(const void* kv_cache, const int32_t* block_table,
                                              const int32_t* key_starts,
                                              const int32_t* out_start_loc, void* latent_out,
                                              void* rope_out, int num_seqs, int num_rows,
                                              int max_blocks_per_seq, int num_blocks,
                                              int latent_size, int rope_size, int block_size,
                                              int kv_dtype, unsigned* device_status,
                                              void* stream) {
  const pattn_status_t v = check_latent_sizes(latent_size, rope_size, block_size, kv_dtype);
  if (v != PATTN_OK) return v;
  if (!kv_cache || !block_table || !out_start_loc || !latent_out || !rope_out)
    return PATTN_ERR_INVALID_ARGUMENT;
  if (num_seqs < 0 || num_rows < 0 || max_blocks_per_seq < 0 || num_blocks < 0)
    return PATTN_ERR_INVALID_ARGUMENT;
  if (misaligned(kv_cache) || misaligned(latent_out) || misaligned(rope_out))
    return PATTN_ERR_INVALID_ARGUMENT;
  if (num_rows == 0 || num_seqs == 0) return PATTN_OK;
  ReadParams p = {};
  p.cache = static_cast<const uint16_t*>(kv_cache);
  p.block_table = block_table;
  p.key_starts = key_starts;
  p.osl = out_start_loc;
  p.latent = static_cast<uint16_t*>(latent_out);
  p.rope = static_cast<uint16_t*>(rope_out);
  p.status = device_status;
  p.B = num_seqs;
  p.rows = num_rows;
  p.mbps = max_blocks_per_seq;
  p.NB = num_blocks;
  p.dc = latent_size;
  p.dr = rope_size;
  p.bs = block_size;
  constexpr long long PER = GL_ROWS * (GL_THREADS / 32);
  const unsigned grid = static_cast<unsigned>((num_rows + PER - 1) / PER);
  return launch_dependent(gather_latent_kernel, dim3(grid), GL_THREADS, 0,
                          static_cast<cudaStream_t>(stream), p) == cudaSuccess
             ? PATTN_OK
             : PATTN_ERR_CUDA;
}
