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
// largest magnitude are log2(LPR) shuffles.  A warp's step serves 32 / LPR rows
// of one token, of one kind (q, k or v).
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
  float eps, inv_d, k_scale, v_scale;
  int T, H, Hkv, D, rot, max_pos, axes, adjacent, vec4;
  int steps_q, steps_kv;   // steps of 32 / LPR rows of a token's q; of its k (and v)
  int stages, stage_bytes;  // ring of the streaming kernel
  int team;                 // warps per token there
  int packed;               // a token's q, k and v rows follow one another
  int bs, NB;
  unsigned char axis[128];  // axis of each rotary pair (axes > 1)
};

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

// (a0, a1) * (b0, b1) + (c0, c1) and (a0, a1) * (b0, b1) on the paired fp32 pipe.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\t"
      "mov.b64 rb, {%4, %5};\n\t"
      "mov.b64 rc, {%6, %7};\n\t"
      "fma.rn.f32x2 rd, ra, rb, rc;\n\t"
      "mov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\t"
      "mov.b64 rb, {%4, %5};\n\t"
      "mul.rn.f32x2 rd, ra, rb;\n\t"
      "mov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// The eight pairs of a lane, a[] and b[], turned: a c - b s, b c + a s.
__device__ __forceinline__ void turn(float (&a)[8], float (&b)[8], const float (&cs)[8],
                                     const float (&sn)[8]) {
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    const float2 a2 = make_float2(a[e], a[e + 1]), b2 = make_float2(b[e], b[e + 1]);
    const float2 c2 = make_float2(cs[e], cs[e + 1]), s2 = make_float2(sn[e], sn[e + 1]);
    const float2 x = fma2(make_float2(-b2.x, -b2.y), s2, mul2(a2, c2));
    const float2 y = fma2(a2, s2, mul2(b2, c2));
    a[e] = x.x;
    a[e + 1] = x.y;
    b[e] = y.x;
    b[e + 1] = y.y;
  }
}

enum RowKind { ROW_Q, ROW_K, ROW_V };

// A lane's place: lane j of the LPR that own a row, and the first elements c0 and
// c1 of its two pieces: of a rotating lane pieces j and j + rot / 16, of the
// others the pieces behind the rotated part, in pairs.
struct LanePlace {
  int j, g, c0, c1;
  bool on, turns;
};
template <int LPR>
__device__ __forceinline__ LanePlace lane_place(const RopeParams& p, int lane) {
  LanePlace l;
  l.j = lane % LPR;
  l.g = lane / LPR;
  const int half = p.rot / 16;  // 8-element pieces of one half of the rotated part
  l.on = l.j < p.D / 16;
  l.turns = l.on && l.j < half;
  l.c0 = (l.turns ? l.j : 2 * l.j) * 8;
  l.c1 = (l.turns ? l.j + half : 2 * l.j + 1) * 8;
  return l;
}

// The cos and sin of a lane's eight pairs: pairs 8j .. 8j + 7 (halves), or, of
// adjacent elements, the four of each piece.  row(a): the table row of the
// token's position on axis a.
template <class Row>
__device__ __forceinline__ void load_turns(const RopeParams& p, const LanePlace& l, Row row,
                                           float (&cs)[8], float (&sn)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int p0 = p.adjacent ? (h ? l.c1 : l.c0) / 2 : 8 * l.j + 4 * h;
    if (p.vec4) {
      const float* r = row(p.axes > 1 ? p.axis[p0] : 0) + p0;
      const float4 c = *reinterpret_cast<const float4*>(r);
      const float4 s = *reinterpret_cast<const float4*>(r + p.rot / 2);
      cs[4 * h] = c.x; cs[4 * h + 1] = c.y; cs[4 * h + 2] = c.z; cs[4 * h + 3] = c.w;
      sn[4 * h] = s.x; sn[4 * h + 1] = s.y; sn[4 * h + 2] = s.z; sn[4 * h + 3] = s.w;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float* r = row(p.axis[p0 + e]) + p0 + e;
        cs[4 * h + e] = r[0];
        sn[4 * h + e] = r[p.rot / 2];
      }
    }
  }
}

// A lane's pieces of a norm's weights.
struct NormWeights {
  uint4 a, b;
  bool on;
};
__device__ __forceinline__ NormWeights norm_weights(const LanePlace& l, const uint16_t* w) {
  NormWeights n;
  n.on = w != nullptr;
  n.a = n.b = make_uint4(0u, 0u, 0u, 0u);
  if (n.on && l.on) {
    n.a = *reinterpret_cast<const uint4*>(w + l.c0);
    n.b = *reinterpret_cast<const uint4*>(w + l.c1);
  }
  return n;
}

// One step of a warp: head h's row of the token (one row per LPR lanes, all of
// one kind; pieces wa and wb) normed, turned and written.  slot: the token's
// cache slot (k and v).  live: the lane has a part of a row that exists.
template <int LPR, int KIND, RowKind R>
__device__ __forceinline__ void serve_row(const RopeParams& p, const LanePlace& l,
                                          const NormWeights& w, const uint4& wa, const uint4& wb,
                                          const float (&cs)[8], const float (&sn)[8], int t, int h,
                                          int64_t slot, bool live) {
  constexpr bool HALF = KIND == PATTN_KV_F16;
  constexpr bool QUANT = KIND == PATTN_KV_FP8_E4M3 || KIND == PATTN_KV_FP8_E4M3_ROW;
  float x[8], y[8];
  unpack8<HALF>(wa, x);
  unpack8<HALF>(wb, y);
  if (R != ROW_V && w.on) {
    float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const float2 a = make_float2(x[e], x[e + 1]), b = make_float2(y[e], y[e + 1]);
      s2 = fma2(b, b, fma2(a, a, s2));
    }
    float ss = s2.x + s2.y;
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float r = rsqrtf(ss * p.inv_d + p.eps);
    const float2 r2 = make_float2(r, r);
    float wx[8], wy[8];
    unpack8<HALF>(w.a, wx);
    unpack8<HALF>(w.b, wy);
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const float2 a = mul2(make_float2(x[e], x[e + 1]), mul2(r2, make_float2(wx[e], wx[e + 1])));
      const float2 b = mul2(make_float2(y[e], y[e + 1]), mul2(r2, make_float2(wy[e], wy[e + 1])));
      x[e] = a.x;
      x[e + 1] = a.y;
      y[e] = b.x;
      y[e + 1] = b.y;
    }
  }
  if (R != ROW_V && l.turns) {
    if (p.adjacent) {
      float a[8], b[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        a[e] = x[2 * e];
        b[e] = x[2 * e + 1];
        a[4 + e] = y[2 * e];
        b[4 + e] = y[2 * e + 1];
      }
      turn(a, b, cs, sn);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[2 * e] = a[e];
        x[2 * e + 1] = b[e];
        y[2 * e] = a[4 + e];
        y[2 * e + 1] = b[4 + e];
      }
    } else {
      turn(x, y, cs, sn);
    }
  }
  if constexpr (R == ROW_Q) {
    if (live) {
      uint16_t* d = p.q_out + t * p.qo_stride + h * p.D;
      *reinterpret_cast<uint4*>(d + l.c0) = pack8<HALF>(x);
      *reinterpret_cast<uint4*>(d + l.c1) = pack8<HALF>(y);
    }
  } else {
    constexpr int kv = R == ROW_V ? 1 : 0;
    const int64_t dst = ((static_cast<int64_t>(kv) * p.NB * p.bs + slot) * p.Hkv + h) * p.D;
    if constexpr (QUANT) {
      float scale = kv ? p.v_scale : p.k_scale;
      if constexpr (KIND == PATTN_KV_FP8_E4M3_ROW) {
        // the row's largest magnitude (NaN elements do not count)
        float m = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = fmaxf(m, fmaxf(fabsf(x[e]), fabsf(y[e])));
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        scale = fminf(fmaxf(__fdiv_rn(m, E4M3_MAX), PATTN_ROW_SCALE_MIN), PATTN_ROW_SCALE_MAX);
      }
      if (live) {
        unsigned char* d = static_cast<unsigned char*>(p.cache) + dst;
        *reinterpret_cast<uint2*>(d + l.c0) = codes8(x, scale);
        *reinterpret_cast<uint2*>(d + l.c1) = codes8(y, scale);
        // slot = block * bs + offset, so slot / 16 counts the groups of 16 slots
        if constexpr (KIND == PATTN_KV_FP8_E4M3_ROW)
          if (l.j == 0)
            p.row_scales[((slot >> 4) * p.Hkv + h) * 32 + kv * 16 + (slot & 15)] = scale;
      }
    } else if (live) {
      uint16_t* d = static_cast<uint16_t*>(p.cache) + dst;
      *reinterpret_cast<uint4*>(d + l.c0) = pack8<HALF>(x);
      *reinterpret_cast<uint4*>(d + l.c1) = pack8<HALF>(y);
    }
  }
}

// ------------------------------------------------------------- few tokens
// One warp per step (latency: every load of the call is in flight at once).
// 1 token of 32 + 2 x 8 heads of 128: 2.6 us, an empty launch's time.
template <int LPR, int KIND>
__global__ void __launch_bounds__(RC_THREADS)
    rope_few_kernel(const __grid_constant__ RopeParams p) {
  constexpr int RPS = 32 / LPR;  // rows per step
  const int steps = p.steps_q + 2 * p.steps_kv;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * (RC_THREADS / 32) + (threadIdx.x >> 5);
  const int t = static_cast<int>(unit / steps);
  if (t >= p.T) return;
  const int step = static_cast<int>(unit - static_cast<int64_t>(t) * steps);
  const int lane = threadIdx.x & 31;
  const LanePlace l = lane_place<LPR>(p, lane);
  int i = step;
  const RowKind kind = i < p.steps_q ? ROW_Q : i < p.steps_q + p.steps_kv ? ROW_K : ROW_V;
  i -= kind == ROW_Q ? 0 : kind == ROW_K ? p.steps_q : p.steps_q + p.steps_kv;
  const int h = i * RPS + l.g;
  const bool live = l.on && h < (kind == ROW_Q ? p.H : p.Hkv);
  uint4 wa = make_uint4(0u, 0u, 0u, 0u), wb = wa;
  if (live) {
    const uint16_t* src = (kind == ROW_Q   ? p.q + t * p.q_stride
                           : kind == ROW_K ? p.key + t * p.k_stride
                                           : p.value + t * p.v_stride) +
                          h * p.D;
    wa = *reinterpret_cast<const uint4*>(src + l.c0);
    wb = *reinterpret_cast<const uint4*>(src + l.c1);
  }
  int64_t slot = 0;
  if (kind != ROW_Q) slot = p.slots[t];
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
      if (pos[0] >= 0 && step == 0 && lane == 0) flag_status(p.status, PATTN_DEV_BAD_METADATA);
      return;
    }
    if (l.turns && kind != ROW_V)
      load_turns(p, l, [&](int a) {
        return p.table + (a == 0 ? pos[0] : a == 1 ? pos[1] : a == 2 ? pos[2] : pos[3]) * p.rot;
      }, cs, sn);
  }
  if (kind != ROW_Q && slot >= static_cast<int64_t>(p.NB) * p.bs) {
    if (step == p.steps_q && lane == 0) flag_status(p.status, PATTN_DEV_BAD_METADATA);
    return;
  }
  if (slot < 0) return;
  const NormWeights w = norm_weights(l, kind == ROW_Q ? p.q_norm : kind == ROW_K ? p.k_norm : nullptr);
  if (kind == ROW_Q) serve_row<LPR, KIND, ROW_Q>(p, l, w, wa, wb, cs, sn, t, h, slot, live);
  else if (kind == ROW_K) serve_row<LPR, KIND, ROW_K>(p, l, w, wa, wb, cs, sn, t, h, slot, live);
  else serve_row<LPR, KIND, ROW_V>(p, l, w, wa, wb, cs, sn, t, h, slot, live);
}

// ------------------------------------------------------------- many tokens
// Persistent CTAs stream their tokens through a ring of shared-memory stages:
// a producer warp reads positions and slots 32 tokens at a time and copies each
// token's q, k and v rows and table rows with untiled bulk copies (one for the
// rows of a packed projection, q, k and v side by side), up to a ring of them
// ahead.  The bytes in flight then depend on the ring, not on what the warps'
// registers hold.  Eight consumer warps work in teams of two, four or eight, a
// team per token: the smaller, the more rows share a warp's cos, sin and norm
// weights, the larger, the fewer stages the teams hold.
// 8384 tokens, 64 q and 8 k and v heads of 128, row-scaled e4m3 cache: 56 us,
// 87 % of the measured copy bandwidth (teams of 8 / 4 / 2 warps 62 / 56.5 / 56).
// 5003 tokens, 32 and 4 heads, norm, three axes: 24.7 us (30.6 / 26.4 / 24.6).
// A second producer warp: 60 and 23.8.
constexpr int RS_WARPS = 8;  // consumer warps
constexpr int RS_STAGES_MAX = 8;
constexpr int RS_RING_BYTES = 100 * 1024;  // two CTAs per SM
constexpr int RS_HEAD = 256;               // barriers and the stages' tokens
constexpr long long RS_LEAST_STAGE = 4096;        // bytes of a token that streaming pays for
constexpr long long RS_LEAST_CALL = 28ll << 20;   // and of a call

struct StreamHead {
  uint64_t full[RS_STAGES_MAX], empty[RS_STAGES_MAX];
  int64_t slot[RS_STAGES_MAX];  // the stage's token: its cache slot, -1 for none
  int token[RS_STAGES_MAX];     // and index; -1: no more tokens
};
static_assert(sizeof(StreamHead) <= RS_HEAD, "the ring's head fits the space kept for it");

template <int LPR, int KIND>
__global__ void __launch_bounds__((RS_WARPS + 1) * 32, 2)
    rope_stream_kernel(const __grid_constant__ RopeParams p) {
  constexpr int RPS = 32 / LPR;
  extern __shared__ __align__(128) unsigned char smem[];
  StreamHead* hd = reinterpret_cast<StreamHead*>(smem);
  unsigned char* ring = smem + RS_HEAD;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q_bytes = p.H * p.D * 2, kv_bytes = p.Hkv * p.D * 2;
  const int row_bytes = p.rot * 4;
  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&hd->full[i], 1);
      mbar_init(&hd->empty[i], p.team);
    }
    fence_mbar_init();
  }
  __syncthreads();

  if (warp == RS_WARPS) {
    // ---------------------------------------------------------- producer
    int n = 0;  // stages filled so far
    bool ok = true;
    auto stage_free = [&]() {
      return n < p.stages || mbar_wait(&hd->empty[n % p.stages], ((n / p.stages) - 1) & 1, p.status,
                                       nullptr);
    };
    for (int64_t base = blockIdx.x; ok && base < p.T; base += 32LL * gridDim.x) {
      const int64_t mine = base + static_cast<int64_t>(lane) * gridDim.x;
      int64_t slot = -1;
      int pos[4] = {0, 0, 0, 0};
      bool skip = mine >= p.T;
      if (!skip) {
        // as in rope_few_kernel: padding and bad tokens
        bool bad = false, padding = false;
#pragma unroll
        for (int a = 0; a < 4; ++a) {
          const int64_t x = a < p.axes ? p.positions[a * p.pos_stride + mine] : 0;
          bad |= x < 0 || x >= p.max_pos;
          if (a == 0) padding = x < 0;
          pos[a] = static_cast<int>(x);
        }
        skip = p.axes > 0 && bad;
        if (skip && !padding) flag_status(p.status, PATTN_DEV_BAD_METADATA);
        if (p.Hkv > 0 && !skip) {
          slot = p.slots[mine];
          if (slot >= static_cast<int64_t>(p.NB) * p.bs) {
            flag_status(p.status, PATTN_DEV_BAD_METADATA);
            slot = -1;
          }
        }
      }
      if (p.H == 0 && slot < 0) skip = true;  // nothing to write
      unsigned todo = __ballot_sync(0xffffffffu, !skip);
      while (ok && todo) {
        const int from = __ffs(todo) - 1;
        todo &= todo - 1;
        const int t = static_cast<int>(base + static_cast<int64_t>(from) * gridDim.x);
        const int64_t s = __shfl_sync(0xffffffffu, slot, from);
        int at[4];
#pragma unroll
        for (int a = 0; a < 4; ++a) at[a] = __shfl_sync(0xffffffffu, pos[a], from);
        if (lane == 0) {
          ok = stage_free();
          if (ok) {
            const int st = n % p.stages;
            unsigned char* d = ring + st * p.stage_bytes;
            hd->token[st] = t;
            hd->slot[st] = s;
            const int kvb = s >= 0 ? kv_bytes : 0;
            mbar_arrive_expect_tx(&hd->full[st], q_bytes + 2 * kvb + p.axes * row_bytes);
            if (q_bytes)
              bulk_load(d, p.q + t * p.q_stride, p.packed ? q_bytes + 2 * kvb : q_bytes,
                        &hd->full[st]);
            if (kvb && !p.packed) {
              bulk_load(d + q_bytes, p.key + t * p.k_stride, kvb, &hd->full[st]);
              bulk_load(d + q_bytes + kv_bytes, p.value + t * p.v_stride, kvb, &hd->full[st]);
            }
#pragma unroll
            for (int a = 0; a < 4; ++a)
              if (a < p.axes)
                bulk_load(d + q_bytes + 2 * kv_bytes + a * row_bytes,
                          p.table + static_cast<int64_t>(at[a]) * p.rot, row_bytes, &hd->full[st]);
          }
        }
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        if (ok) ++n;
      }
    }
    if (lane == 0) {
      // one end mark for each team
      const int end = n + RS_WARPS / p.team;
      for (; ok && n < end; ++n) {
        if (!(ok = stage_free())) break;
        hd->token[n % p.stages] = -1;
        mbar_arrive(&hd->full[n % p.stages]);
      }
      if (!ok) {
        // a wait gave up: no copy may still be writing shared memory at the exit
        drain_armed(hd->full, p.stages, n, -1, p.status);
      }
    }
    return;
  }

  // ------------------------------------------------------------ consumers
  const LanePlace l = lane_place<LPR>(p, lane);
  const NormWeights wq = norm_weights(l, p.q_norm);
  const int steps = p.steps_q + 2 * p.steps_kv;
  const int teams = RS_WARPS / p.team, me = warp % p.team;
  for (int n = warp / p.team;; n += teams) {
    const int st = n % p.stages;
    if (!__all_sync(0xffffffffu, mbar_wait(&hd->full[st], (n / p.stages) & 1, p.status, nullptr)))
      return;
    const int t = *static_cast<volatile int*>(&hd->token[st]);
    if (t < 0) return;
    const int64_t slot = *static_cast<volatile int64_t*>(&hd->slot[st]);
    const unsigned char* d = ring + st * p.stage_bytes;
    float cs[8], sn[8];
    if (l.turns) {
      const float* rows = reinterpret_cast<const float*>(d + q_bytes + 2 * kv_bytes);
      load_turns(p, l, [&](int a) { return rows + a * p.rot; }, cs, sn);
    }
    // the members' shares of the steps move on by one with each token
    const int end = slot >= 0 ? steps : p.steps_q;
    for (int i = (me + n) % p.team; i < end; i += p.team) {
      const bool is_q = i < p.steps_q, is_k = !is_q && i < p.steps_q + p.steps_kv;
      const int h = (i - (is_q ? 0 : is_k ? p.steps_q : p.steps_q + p.steps_kv)) * RPS + l.g;
      const bool live = l.on && h < (is_q ? p.H : p.Hkv);
      uint4 wa = make_uint4(0u, 0u, 0u, 0u), wb = wa;
      if (live) {
        const unsigned char* src = d + (is_q ? 0 : is_k ? q_bytes : q_bytes + kv_bytes) + h * p.D * 2;
        wa = *reinterpret_cast<const uint4*>(src + l.c0 * 2);
        wb = *reinterpret_cast<const uint4*>(src + l.c1 * 2);
      }
      if (is_q) serve_row<LPR, KIND, ROW_Q>(p, l, wq, wa, wb, cs, sn, t, h, slot, live);
      else if (is_k)
        serve_row<LPR, KIND, ROW_K>(p, l, norm_weights(l, p.k_norm), wa, wb, cs, sn, t, h, slot, live);
      else serve_row<LPR, KIND, ROW_V>(p, l, wq, wa, wb, cs, sn, t, h, slot, live);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&hd->empty[st]);
  }
}

template <int LPR, int KIND>
cudaError_t launch_kind(RopeParams& p, int sms, cudaStream_t st) {
  const long long steps = p.steps_q + 2LL * p.steps_kv;
  const long long stage = (2LL * (p.H + 2LL * p.Hkv) * p.D + 4LL * p.axes * p.rot + 127) / 128 * 128;
  // Stream long calls of tokens with long rows (in us, one warp per step against
  // streamed): 64 + 2 x 8 heads of 128, 608 tokens 7.2 / 6.7, 1216 14.4 / 13.9,
  // 8384 77 / 56; 32 + 2 x 8, 1824 tokens 13.2 / 14.5, 2432 17.1 / 16.7, 4864
  // 30.0 / 26.1; 16 + 2 x 2 of 128, 3000 tokens 11.0 / 11.7, 6000 21.0 / 19.3;
  // of 64, 3000 tokens 8.0 / 9.8, 24000 53 / 58 (a copy's cost shows).  One count
  // of bytes for all widths: it keeps 32 heads off the slower side and costs calls
  // of 64 heads below it half a microsecond.  And the ring has to hold three tokens.
  if (stage >= RS_LEAST_STAGE && p.T * stage >= RS_LEAST_CALL && 3 * stage <= RS_RING_BYTES) {
    p.stage_bytes = static_cast<int>(stage);
    p.packed = p.H > 0 && p.Hkv > 0 && p.key == p.q + p.H * p.D && p.value == p.key + p.Hkv * p.D &&
               p.q_stride == p.k_stride && p.q_stride == p.v_stride;
    p.stages = static_cast<int>(std::min<long long>(RS_STAGES_MAX, RS_RING_BYTES / stage));
    // the smallest team that leaves the producer as many stages as the teams hold
    // (two warps at least: teams of one would need sixteen)
    p.team = RS_WARPS;
    while (p.team > 1 && 2 * (2 * RS_WARPS / p.team) <= p.stages) p.team /= 2;
    const int smem = RS_HEAD + p.stages * p.stage_bytes;
    auto kern = rope_stream_kernel<LPR, KIND>;
    // The limit belongs to the kernel, not to this launch: the same value in every
    // call, so that no host thread lowers it between another's set and launch.
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               RS_HEAD + RS_RING_BYTES);
    if (e != cudaSuccess) return e;
    kern<<<2 * sms, (RS_WARPS + 1) * 32, smem, st>>>(p);
  } else {
    const long long ctas = (p.T * steps + RC_THREADS / 32 - 1) / (RC_THREADS / 32);
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    rope_few_kernel<LPR, KIND><<<static_cast<unsigned>(ctas), RC_THREADS, 0, st>>>(p);
  }
  return cudaGetLastError();
}

template <int LPR>
cudaError_t launch_lpr(RopeParams& p, int kv_dtype, int sms, cudaStream_t st) {
  p.steps_q = (p.H + 32 / LPR - 1) / (32 / LPR);
  p.steps_kv = (p.Hkv + 32 / LPR - 1) / (32 / LPR);
  switch (kv_dtype) {
    case PATTN_KV_F16: return launch_kind<LPR, PATTN_KV_F16>(p, sms, st);
    case PATTN_KV_FP8_E4M3: return launch_kind<LPR, PATTN_KV_FP8_E4M3>(p, sms, st);
    case PATTN_KV_FP8_E4M3_ROW: return launch_kind<LPR, PATTN_KV_FP8_E4M3_ROW>(p, sms, st);
    default: return launch_kind<LPR, PATTN_KV_BF16>(p, sms, st);
  }
}

pattn_status_t launch(RopeParams& p, int kv_dtype, cudaStream_t st) {
  const int sms = current_sms();
  const cudaError_t e = p.D <= 64    ? launch_lpr<4>(p, kv_dtype, sms, st)
                        : p.D <= 128 ? launch_lpr<8>(p, kv_dtype, sms, st)
                                     : launch_lpr<16>(p, kv_dtype, sms, st);
  return e == cudaSuccess ? PATTN_OK : PATTN_ERR_CUDA;
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
  p.inv_d = 1.f / static_cast<float>(D);
  p.rot = a->num_axes > 0 ? rot : 0;
  p.max_pos = a->max_position;
  p.axes = a->num_axes;
  p.adjacent = a->interleaved;
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
