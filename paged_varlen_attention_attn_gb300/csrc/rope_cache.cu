// rope_cache.cu -- rotary embedding of new tokens and their (quantising) cache
// write in one pass (sm_103a).
//
// For each token: q and k heads are optionally normed,
//   x <- x * rsqrt(mean(x^2) + eps) * w,
// and rotated: rotary pair p of a head, (a, b), becomes
//   (a cos - b sin, b cos + a sin),  angle = pos[axis(p)] * frequency_p,
// with cos and sin from an fp32 table whose row is a position.  One position
// per token (one axis), or one per axis (time, height, width) with a table
// that says which axis turns which pair.  q goes to q_out; k (rotated) and v
// go to the paged cache: as they are, as e4m3 of one scale per tensor, or as
// e4m3 with one scale per (token, KV head) row,
//   s = clamp(max|x| / 448, 2^-60, 2^60), code = e4m3(x / s).
// Everything between the 16-bit inputs and the one rounding of the output is
// fp32: nothing is rounded between norm, rotation and quantisation.
//
// Bound by HBM: every byte is read once and written once.  LPR = 4 / 8 / 16
// lanes own one head row (head sizes up to 64 / 128 / 256), 16 elements each
// as two 16-byte pieces: the two pieces that a rotation in halves pairs up, so
// a lane holds both elements of its eight pairs and a row's sum of squares and
// largest magnitude are log2(LPR) shuffles.  A warp serves 32 / LPR rows of
// one token at a time and walks the token's rows, so the eight cos and sin
// values of its lanes are loaded once, and the next rows' pieces load while
// the current ones are worked on.
#include <algorithm>
#include <cmath>

#include "../../include/pattn.h"
#include "common.cuh"
#include "internal.h"

namespace pattn {
namespace {

constexpr int RC_THREADS = 128;
constexpr float E4M3_MAX = 448.f;

struct RopeParams {
  const uint16_t* q;
  uint16_t* q_out;
  const uint16_t* key;
  const uint16_t* value;
  int64_t q_stride, qo_stride, k_stride, v_stride;  // elements between tokens
  const float* table;                               // [max_pos][rot]: cos, then sin
  const int64_t* positions;                         // [axes][pos_stride]
  int64_t pos_stride;
  const uint16_t* q_norm;
  const uint16_t* k_norm;
  const int64_t* slots;
  void* cache;
  float* row_scales;
  unsigned* status;
  float eps, k_scale, v_scale;
  int T, H, Hkv, D, rot, max_pos, axes, adjacent, vec4;
  int nq, rows;            // q rows of a token (0 without q), all its rows
  int chunks, iters;       // warps per token, steps of 32 / LPR rows each takes
  int bs, NB;
  unsigned char axis[128];  // axis of each rotary pair (axes > 1)
};

template <bool HALF>
__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  const unsigned u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (HALF) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    } else {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
}

template <bool HALF>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack2<HALF>(x[0], x[1]), pack2<HALF>(x[2], x[3]), pack2<HALF>(x[4], x[5]),
                    pack2<HALF>(x[6], x[7]));
}

// Eight values over their scale as e4m3 codes: the fp32 quotient, as in
// pattn_reshape_and_cache, rounded to nearest even, saturated at +-448, NaN
// kept.
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float sc) {
  unsigned w[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = make_float2(__fdiv_rn(x[2 * i], sc), __fdiv_rn(x[2 * i + 1], sc));
    const unsigned c = __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
    w[i >> 1] |= c << ((i & 1) * 16);
  }
  return make_uint2(w[0], w[1]);
}

// LPR: lanes per row.  KIND: the cache (PATTN_KV_*); f16 data goes with KIND
// PATTN_KV_F16, bf16 data with every other.
template <int LPR, int KIND>
__global__ void __launch_bounds__(RC_THREADS)
    rope_cache_kernel(const __grid_constant__ RopeParams p) {
  constexpr bool HALF = KIND == PATTN_KV_F16;
  constexpr bool QUANT = KIND == PATTN_KV_FP8_E4M3 || KIND == PATTN_KV_FP8_E4M3_ROW;
  constexpr int RPS = 32 / LPR;  // rows per step of a warp
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * (RC_THREADS / 32) + (threadIdx.x >> 5);
  const int t = static_cast<int>(unit / p.chunks);
  if (t >= p.T) return;
  const int chunk = static_cast<int>(unit - static_cast<int64_t>(t) * p.chunks);
  const int lane = threadIdx.x & 31;
  const int j = lane % LPR, g = lane / LPR;
  const int half = p.rot / 16;      // 8-element pieces of one half of the rotated part
  const bool lane_on = j < p.D / 16;
  const bool turns = lane_on && j < half;
  // this lane's two pieces: a rotating lane's j and j + half, then pairs of
  // pieces behind the rotated part
  const int c0 = turns ? j : 2 * j, c1 = turns ? j + half : 2 * j + 1;

  // row `row` of the token: q heads, then k heads, then v heads
  const int row0 = chunk * p.iters * RPS + g;
  const int row_end = min(p.rows, (chunk + 1) * p.iters * RPS);
  auto src_of = [&](int row) -> const uint16_t* {
    if (row < p.nq) return p.q + t * p.q_stride + static_cast<int64_t>(row) * p.D;
    row -= p.nq;
    return row < p.Hkv ? p.key + t * p.k_stride + static_cast<int64_t>(row) * p.D
                       : p.value + t * p.v_stride + static_cast<int64_t>(row - p.Hkv) * p.D;
  };
  auto load = [&](int row, uint4& a, uint4& b) {
    a = b = make_uint4(0u, 0u, 0u, 0u);
    if (lane_on && row < row_end) {
      const uint16_t* s = src_of(row);
      a = *reinterpret_cast<const uint4*>(s + c0 * 8);
      b = *reinterpret_cast<const uint4*>(s + c1 * 8);
    }
  };
  // two steps' rows are in flight while the positions and the table load
  uint4 na0, nb0, na1, nb1;
  load(row0, na0, nb0);
  load(row0 + RPS, na1, nb1);

  // The token's positions: a negative first one marks padding (nothing of the
  // token is written), any other outside the table is reported and skipped.
  float cs[8], sn[8];
  if (p.axes > 0) {
    int64_t pos[4];
    bool bad = false;
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      pos[a] = a < p.axes ? p.positions[a * p.pos_stride + t] : 0;
      bad |= pos[a] < 0 || pos[a] >= p.max_pos;
    }
    if (bad) {
      if (pos[0] >= 0 && chunk == 0 && lane == 0) flag_status(p.status, PATTN_DEV_BAD_METADATA);
      return;
    }
    if (turns) {
      // pairs of the lane: 8j .. 8j + 7 (halves), or, of adjacent elements,
      // the four of each piece
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int p0 = p.adjacent ? 4 * (h ? c1 : c0) : 8 * j + 4 * h;
        if (p.vec4) {
          const int a = p.axes > 1 ? p.axis[p0] : 0;
          const int64_t at = a == 0 ? pos[0] : a == 1 ? pos[1] : a == 2 ? pos[2] : pos[3];
          const float* trow = p.table + at * p.rot + p0;
          const float4 c = *reinterpret_cast<const float4*>(trow);
          const float4 s = *reinterpret_cast<const float4*>(trow + p.rot / 2);
          cs[4 * h] = c.x; cs[4 * h + 1] = c.y; cs[4 * h + 2] = c.z; cs[4 * h + 3] = c.w;
          sn[4 * h] = s.x; sn[4 * h + 1] = s.y; sn[4 * h + 2] = s.z; sn[4 * h + 3] = s.w;
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int a = p.axis[p0 + e];
            const int64_t at = a == 0 ? pos[0] : a == 1 ? pos[1] : a == 2 ? pos[2] : pos[3];
            cs[4 * h + e] = p.table[at * p.rot + p0 + e];
            sn[4 * h + e] = p.table[at * p.rot + p.rot / 2 + p0 + e];
          }
        }
      }
    }
  }
  // Where the token's key and value rows go; -1: nowhere.
  int64_t blk = -1;
  int off = 0;
  if (p.Hkv > 0) {
    const int64_t s = p.slots[t];
    if (s >= static_cast<int64_t>(p.NB) * p.bs) {
      if (chunk == 0 && lane == 0) flag_status(p.status, PATTN_DEV_BAD_METADATA);
    } else if (s >= 0) {
      blk = s / p.bs;
      off = static_cast<int>(s - blk * p.bs);
    }
  }
  const bool normed = p.q_norm != nullptr || p.k_norm != nullptr;
  const float inv_d = 1.f / static_cast<float>(p.D);

  for (int i = 0; i < p.iters; ++i) {
    const int row = row0 + i * RPS;
    const uint4 wa = na0, wb = nb0;
    na0 = na1;
    nb0 = nb1;
    load(row + 2 * RPS, na1, nb1);
    const bool live = row < row_end;
    const int kind = row < p.nq ? 0 : row < p.nq + p.Hkv ? 1 : 2;  // q, k, v
    float x[8], y[8];
    unpack8<HALF>(wa, x);
    unpack8<HALF>(wb, y);
    if (normed) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss += x[e] * x[e] + y[e] * y[e];
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const uint16_t* w = kind == 0 ? p.q_norm : kind == 1 ? p.k_norm : nullptr;
      if (w && lane_on) {
        const float r = rsqrtf(ss * inv_d + p.eps);
        float wx[8], wy[8];
        unpack8<HALF>(*reinterpret_cast<const uint4*>(w + c0 * 8), wx);
        unpack8<HALF>(*reinterpret_cast<const uint4*>(w + c1 * 8), wy);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[e] *= r * wx[e];
          y[e] *= r * wy[e];
        }
      }
    }
    if (p.axes > 0 && kind < 2 && turns) {
      if (p.adjacent) {
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
    }
    float scale = kind == 1 ? p.k_scale : p.v_scale;
    if constexpr (KIND == PATTN_KV_FP8_E4M3_ROW) {
      // the row's largest magnitude (NaN elements do not count)
      float m = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) m = fmaxf(m, fmaxf(fabsf(x[e]), fabsf(y[e])));
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      scale = fminf(fmaxf(__fdiv_rn(m, E4M3_MAX), PATTN_ROW_SCALE_MIN), PATTN_ROW_SCALE_MAX);
    }
    if (!live || !lane_on) continue;
    if (kind == 0) {
      uint16_t* d = p.q_out + t * p.qo_stride + static_cast<int64_t>(row) * p.D;
      *reinterpret_cast<uint4*>(d + c0 * 8) = pack8<HALF>(x);
      *reinterpret_cast<uint4*>(d + c1 * 8) = pack8<HALF>(y);
      continue;
    }
    if (blk < 0) continue;
    const int kv = kind - 1, h = row - p.nq - kv * p.Hkv;
    const int64_t dst =
        (((static_cast<int64_t>(kv) * p.NB + blk) * p.bs + off) * p.Hkv + h) * p.D;
    if constexpr (QUANT) {
      unsigned char* d = static_cast<unsigned char*>(p.cache) + dst;
      *reinterpret_cast<uint2*>(d + c0 * 8) = codes8(x, scale);
      *reinterpret_cast<uint2*>(d + c1 * 8) = codes8(y, scale);
      if constexpr (KIND == PATTN_KV_FP8_E4M3_ROW)
        if (j == 0)
          p.row_scales[((blk * (p.bs / 16) + (off >> 4)) * p.Hkv + h) * 32 + kv * 16 + (off & 15)] =
              scale;
    } else {
      uint16_t* d = static_cast<uint16_t*>(p.cache) + dst;
      *reinterpret_cast<uint4*>(d + c0 * 8) = pack8<HALF>(x);
      *reinterpret_cast<uint4*>(d + c1 * 8) = pack8<HALF>(y);
    }
  }
}

template <int LPR>
void launch_lpr(const RopeParams& p, int kv_dtype, unsigned grid, cudaStream_t st) {
  switch (kv_dtype) {
    case PATTN_KV_F16: rope_cache_kernel<LPR, PATTN_KV_F16><<<grid, RC_THREADS, 0, st>>>(p); break;
    case PATTN_KV_FP8_E4M3:
      rope_cache_kernel<LPR, PATTN_KV_FP8_E4M3><<<grid, RC_THREADS, 0, st>>>(p);
      break;
    case PATTN_KV_FP8_E4M3_ROW:
      rope_cache_kernel<LPR, PATTN_KV_FP8_E4M3_ROW><<<grid, RC_THREADS, 0, st>>>(p);
      break;
    default: rope_cache_kernel<LPR, PATTN_KV_BF16><<<grid, RC_THREADS, 0, st>>>(p); break;
  }
}

// Fills in how the rows are dealt out and launches.  Few tokens: one step per
// warp (all rows at once, latency); many: up to MAX_ITERS steps per warp, so
// that the cos and sin loads are shared, once that still leaves WARPS_WANTED.
pattn_status_t launch(RopeParams& p, int kv_dtype, cudaStream_t st) {
  constexpr long long WARPS_WANTED = 152 * 32;
  constexpr int MAX_ITERS = 10;
  const int lpr = p.D <= 64 ? 4 : p.D <= 128 ? 8 : 16;
  const int steps = (p.rows + 32 / lpr - 1) / (32 / lpr);
  const long long all = static_cast<long long>(p.T) * steps;
  p.iters = static_cast<int>(
      std::max(1LL, std::min<long long>(std::min(MAX_ITERS, steps), all / WARPS_WANTED)));
  p.chunks = (steps + p.iters - 1) / p.iters;
  const long long ctas = (static_cast<long long>(p.T) * p.chunks + RC_THREADS / 32 - 1) /
                         (RC_THREADS / 32);
  if (ctas > 0x7fffffffLL) return PATTN_ERR_UNSUPPORTED;
  const unsigned grid = static_cast<unsigned>(ctas);
  if (lpr == 4) launch_lpr<4>(p, kv_dtype, grid, st);
  else if (lpr == 8) launch_lpr<8>(p, kv_dtype, grid, st);
  else launch_lpr<16>(p, kv_dtype, grid, st);
  return cudaGetLastError() == cudaSuccess ? PATTN_OK : PATTN_ERR_CUDA;
}

bool misaligned(const void* x) { return (reinterpret_cast<uintptr_t>(x) & 15) != 0; }

}  // namespace
}  // namespace pattn

using namespace pattn;

extern "C" pattn_status_t pattn_rope_and_cache(const pattn_rope_t* a) {
  if (!a || a->struct_size < sizeof(pattn_rope_t)) return PATTN_ERR_INVALID_ARGUMENT;
  const bool has_q = a->q != nullptr, has_kv = a->key != nullptr;
  if (!has_q && !has_kv) return PATTN_ERR_INVALID_ARGUMENT;
  if (has_q != (a->q_out != nullptr) || has_kv != (a->value != nullptr))
    return PATTN_ERR_INVALID_ARGUMENT;
  if (a->num_tokens < 0) return PATTN_ERR_INVALID_ARGUMENT;
  if (has_q && a->num_heads <= 0) return PATTN_ERR_INVALID_ARGUMENT;
  if (has_kv && (a->num_kv_heads <= 0 || !a->kv_cache || !a->slot_mapping || a->num_blocks < 0 ||
                 a->block_size <= 0 || a->block_size % 16 != 0))
    return PATTN_ERR_INVALID_ARGUMENT;
  const int D = a->head_size, rot = a->rot_dim;
  if (D <= 0 || D % 16 != 0 || D > 256) return PATTN_ERR_UNSUPPORTED;
  if (a->num_axes < 0 || a->num_axes > 4 || (a->interleaved != 0 && a->interleaved != 1))
    return PATTN_ERR_INVALID_ARGUMENT;
  if (a->kv_dtype != PATTN_KV_BF16 && a->kv_dtype != PATTN_KV_FP8_E4M3 &&
      a->kv_dtype != PATTN_KV_F16 && a->kv_dtype != PATTN_KV_FP8_E4M3_ROW)
    return PATTN_ERR_UNSUPPORTED;
  RopeParams p = {};
  if (a->num_axes > 0) {
    if (!a->cos_sin || !a->positions || a->max_position <= 0 || rot <= 0 || rot > D)
      return PATTN_ERR_INVALID_ARGUMENT;
    if (rot % 16 != 0) return PATTN_ERR_UNSUPPORTED;
    if (misaligned(a->cos_sin) || (a->num_axes > 1 && (!a->pair_axis || a->positions_stride < 0)))
      return PATTN_ERR_INVALID_ARGUMENT;
    p.vec4 = 1;
    for (int i = 0; a->num_axes > 1 && i < rot / 2; ++i) {
      if (a->pair_axis[i] >= a->num_axes) return PATTN_ERR_INVALID_ARGUMENT;
      p.axis[i] = a->pair_axis[i];
      if (i % 4 && p.axis[i] != p.axis[i - 1]) p.vec4 = 0;
    }
  }
  if ((a->q_norm || a->k_norm) && !(a->norm_eps >= 0.f && a->norm_eps < INFINITY))
    return PATTN_ERR_INVALID_ARGUMENT;
  if (misaligned(a->q_norm) || misaligned(a->k_norm)) return PATTN_ERR_INVALID_ARGUMENT;
  // rows are moved in 16-byte pieces
  if (has_q && (misaligned(a->q) || misaligned(a->q_out) || a->q_stride % 8 != 0 ||
                a->q_out_stride % 8 != 0))
    return PATTN_ERR_INVALID_ARGUMENT;
  if (has_kv && (misaligned(a->key) || misaligned(a->value) || misaligned(a->kv_cache) ||
                 a->key_stride % 8 != 0 || a->value_stride % 8 != 0))
    return PATTN_ERR_INVALID_ARGUMENT;
  // a token's rows must not reach into the next token's
  const long long q_row = static_cast<long long>(a->num_heads) * D;
  const long long k_row = static_cast<long long>(a->num_kv_heads) * D;
  if (has_q && (a->q_stride < q_row || a->q_out_stride < q_row)) return PATTN_ERR_INVALID_ARGUMENT;
  if (has_kv && (a->key_stride < k_row || a->value_stride < k_row))
    return PATTN_ERR_INVALID_ARGUMENT;
  p.k_scale = p.v_scale = 1.f;
  if (has_kv && a->kv_dtype == PATTN_KV_FP8_E4M3) {
    if (!a->kv_scale || !(a->kv_scale[0] > 0.f) || !(a->kv_scale[1] > 0.f) ||
        !(a->kv_scale[0] < INFINITY) || !(a->kv_scale[1] < INFINITY))
      return PATTN_ERR_INVALID_ARGUMENT;
    p.k_scale = a->kv_scale[0];
    p.v_scale = a->kv_scale[1];
  }
  if (has_kv && a->kv_dtype == PATTN_KV_FP8_E4M3_ROW &&
      (!a->row_scales || misaligned(a->row_scales)))
    return PATTN_ERR_INVALID_ARGUMENT;
  if (a->num_tokens == 0) return PATTN_OK;
  p.q = static_cast<const uint16_t*>(a->q);
  p.q_out = static_cast<uint16_t*>(a->q_out);
  p.key = static_cast<const uint16_t*>(a->key);
  p.value = static_cast<const uint16_t*>(a->value);
  p.q_stride = a->q_stride;
  p.qo_stride = a->q_out_stride;
  p.k_stride = a->key_stride;
  p.v_stride = a->value_stride;
  p.table = a->cos_sin;
  p.positions = a->positions;
  p.pos_stride = a->positions_stride;
  p.q_norm = static_cast<const uint16_t*>(a->q_norm);
  p.k_norm = static_cast<const uint16_t*>(a->k_norm);
  p.eps = a->norm_eps;
  p.slots = a->slot_mapping;
  p.cache = a->kv_cache;
  p.row_scales = a->row_scales;
  p.status = a->device_status;
  p.T = a->num_tokens;
  p.H = has_q ? a->num_heads : 0;
  p.Hkv = has_kv ? a->num_kv_heads : 0;
  p.D = D;
  p.rot = a->num_axes > 0 ? rot : 0;
  p.max_pos = a->max_position;
  p.axes = a->num_axes;
  p.adjacent = a->interleaved;
  p.nq = p.H;
  p.rows = p.H + 2 * p.Hkv;
  p.bs = a->block_size;
  p.NB = a->num_blocks;
  return launch(p, a->kv_dtype, static_cast<cudaStream_t>(a->stream));
}

extern "C" pattn_status_t pattn_reshape_and_cache_rows(
    const void* key, const void* value, void* kv_cache, float* row_scales,
    const int64_t* slot_mapping, int num_tokens, int num_kv_heads, int head_size, int block_size,
    int num_blocks, unsigned* device_status, void* stream) {
  if (!key || !value) return PATTN_ERR_INVALID_ARGUMENT;
  if (num_kv_heads <= 0) return PATTN_ERR_INVALID_ARGUMENT;
  pattn_rope_t a = {};
  a.struct_size = sizeof a;
  a.key = key;
  a.value = value;
  a.key_stride = a.value_stride = static_cast<long long>(num_kv_heads) * head_size;
  a.kv_cache = kv_cache;
  a.row_scales = row_scales;
  a.slot_mapping = slot_mapping;
  a.kv_dtype = PATTN_KV_FP8_E4M3_ROW;
  a.num_tokens = num_tokens;
  a.num_kv_heads = num_kv_heads;
  a.head_size = head_size;
  a.block_size = block_size;
  a.num_blocks = num_blocks;
  a.device_status = device_status;
  a.stream = stream;
  return pattn_rope_and_cache(&a);
}
