// What stands around decode attention: per-head norm and rotation of queries and keys (with its
// gradient), the same written into the paged key-value cache, and the cache read back.
//
//   norm      r = 1 / sqrt(mean_c x_c^2 + eps),  n_c = x_c r w_c
//   rotation  pairs (i, i + R/2), or (2 i, 2 i + 1) interleaved, of the first R channels:
//             y_a = n_a cos_i - n_b sin_i,  y_b = n_b cos_i + n_a sin_i
//   cache     bf16 rows, or e4m3 codes of x / s with s = max(max_c |x_c| / 448, 2^-64) per row
//
// All of it moves each element once or twice and computes little (about 10 flops an element): bound
// by HBM for many tokens, by the launch and two dependent loads for few.  So a row of d channels is
// held by d / 8 lanes (16 or 8), 16 bytes a lane, the norm and the row maximum are shuffles among
// them, and a group of lanes takes four rows (heads) of one token at a time: four loads in flight
// per lane, one read of the token's angles for the four, and one exchange of their four sums.
// Everything is fp32 between the one load and the one rounding; the instructions, not only the
// bytes, count here (90 to 125 per row and lane are half of the issue slots), so the
// products run on packed pairs (f32x2) and the norm's weights are multiplied into the angles.
// 32768 tokens of 96 + 12 heads of 128: 293 us forward, 6.2 TB/s, 95 % of a plain copy's rate; the gradient of
// 4096 tokens 69 us, 4.9 TB/s (two blocks per SM and 180 instructions per row and lane: latency).
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <type_traits>

#include "attn_common.cuh"
#include "kda_device.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;     // of the gradient and the cache read
constexpr int kRopeThreads = 64;  // of the forward: the smaller blocks end more evenly,
constexpr int kRopeCtas = 8;      // this many per SM
constexpr int kRows = 4;          // rows of one token that a group of lanes takes at a time

// Two fp32 values in a 64-bit register, for the packed fp32 instructions.
typedef unsigned long long F2;
__device__ __forceinline__ F2 f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 un2(F2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// Two bf16 as fp32.
__device__ __forceinline__ F2 bf2(uint32_t u) { return f2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u)); }

struct RowVec {
  uint32_t u[4];  // 8 bf16
};
struct Row8 {
  F2 v[4];        // 8 fp32
};

__device__ __forceinline__ RowVec load_row(const __nv_bfloat16* p, bool on) {
  RowVec r;
  // (a plain load: the outputs may be written in place)
  const uint4 t = on ? *reinterpret_cast<const uint4*>(p) : make_uint4(0, 0, 0, 0);
  r.u[0] = t.x; r.u[1] = t.y; r.u[2] = t.z; r.u[3] = t.w;
  return r;
}
__device__ __forceinline__ Row8 to_float(const RowVec& r) {
  Row8 x;
#pragma unroll
  for (int i = 0; i < 4; ++i) x.v[i] = bf2(r.u[i]);
  return x;
}
__device__ __forceinline__ uint32_t pack2(F2 v) {
  const float2 t = un2(v);
  return pack_bf16(t.x, t.y);
}
__device__ __forceinline__ uint4 to_bf16(const Row8& x) { return make_uint4(pack2(x.v[0]), pack2(x.v[1]), pack2(x.v[2]), pack2(x.v[3])); }
// Eight fp32 parameters, or `other` throughout.
__device__ __forceinline__ void load8(const float* p, float (&x)[8], bool on, float other) {
  const float4 a = on ? __ldg(reinterpret_cast<const float4*>(p)) : make_float4(other, other, other, other);
  const float4 b = on ? __ldg(reinterpret_cast<const float4*>(p) + 1) : make_float4(other, other, other, other);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
// The sums of four values over a group of lanes at once: they are halved in number twice while they
// are summed, lane `sub` then holds the total of value 2 (sub / H) + (sub / (H / 2)) % 2, H = kLanes / 2;
// that of value i is lane sum4_lane(i)'s.
template <int kLanes>
__device__ __forceinline__ float sum4(const float (&s)[4]) {
  const int sub = threadIdx.x & (kLanes - 1);
  constexpr int H = kLanes / 2;
  const bool hi = sub & H, lo = sub & (H / 2);
  const float t0 = (hi ? s[2] : s[0]) + __shfl_xor_sync(0xffffffffu, hi ? s[0] : s[2], H);
  const float t1 = (hi ? s[3] : s[1]) + __shfl_xor_sync(0xffffffffu, hi ? s[1] : s[3], H);
  float u = (lo ? t1 : t0) + __shfl_xor_sync(0xffffffffu, lo ? t0 : t1, H / 2);
#pragma unroll
  for (int o = H / 4; o > 0; o >>= 1) u += __shfl_xor_sync(0xffffffffu, u, o);
  return u;
}
template <int kLanes>
__device__ __forceinline__ int sum4_lane(int i) {
  return ((threadIdx.x & 31) & ~(kLanes - 1)) + (i >> 1) * (kLanes / 2) + (i & 1) * (kLanes / 4);
}
template <int kLanes>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// The rotation (kBack: its transpose) of one lane's 8 channels, as y = x own + other cross, where
// `other` are the channels they pair with: the partner lane's of the half-split pairs, the same lane's
// neighbours of the interleaved ones.  With weights w (own channels) and wp (the others') multiplied in.
struct Angles {
  F2 own[4], cross[4];
  int partner;    // lane of the warp
  uint32_t up, high;  // 2^16 and the upper half's mask; 0 where nothing is rotated: an infinity there must
                      // not meet the zero in `cross`
};

template <int kLanes, bool kBack>
__device__ __forceinline__ void load_angles(Angles& g, const float* row, int rot, int interleaved, const float* weight, bool lane_on) {
  const int lane = threadIdx.x & 31, sub = lane & (kLanes - 1);
  const bool on = row != nullptr && 8 * sub < rot;
  const bool second = on && !interleaved && 8 * sub >= rot / 2;
  g.up = on ? 65536u : 0u;
  g.high = on ? 0xffff0000u : 0u;
  g.partner = on && !interleaved ? (second ? lane - rot / 16 : lane + rot / 16) : lane;
  float c[8], s[8], w[8];
  load8(weight + 8 * sub, w, weight != nullptr && lane_on, 1.f);
  if (!on) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      g.own[i] = f2(w[2 * i], w[2 * i + 1]);
      g.cross[i] = f2(0.f, 0.f);
    }
    return;
  }
  if (interleaved) {
    const float4 c4 = __ldg(reinterpret_cast<const float4*>(row + 4 * sub));
    const float4 s4 = __ldg(reinterpret_cast<const float4*>(row + rot / 2 + 4 * sub));
    c[0] = c[1] = c4.x; c[2] = c[3] = c4.y; c[4] = c[5] = c4.z; c[6] = c[7] = c4.w;
    s[0] = s[1] = s4.x; s[2] = s[3] = s4.y; s[4] = s[5] = s4.z; s[6] = s[7] = s4.w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // y_a = x_a c - x_b s, y_b = x_b c + x_a s (transposed: the sines' signs exchanged)
      const float wa = w[2 * i], wb = w[2 * i + 1], sn = kBack ? -s[2 * i] : s[2 * i];
      g.own[i] = f2(c[2 * i] * wa, c[2 * i] * wb);
      g.cross[i] = f2(-sn * wb, sn * wa);
    }
  } else {
    const int at = 8 * sub - (second ? rot / 2 : 0);
    float wp[8];
    load8(row + at, c, true, 0.f);
    load8(row + rot / 2 + at, s, true, 0.f);
    load8(weight + 8 * (g.partner & (kLanes - 1)), wp, weight != nullptr, 1.f);
    const float sign = second != kBack ? 1.f : -1.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      g.own[i] = f2(c[2 * i] * w[2 * i], c[2 * i + 1] * w[2 * i + 1]);
      g.cross[i] = f2(sign * s[2 * i] * wp[2 * i], sign * s[2 * i + 1] * wp[2 * i + 1]);
    }
  }
}
// The channels that a row's rotation pairs with this lane's.
__device__ __forceinline__ Row8 paired(const RowVec& raw, const Angles& g, int interleaved) {
  Row8 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t u = interleaved ? raw.u[i] : __shfl_sync(0xffffffffu, raw.u[i], g.partner);
    const float first = __uint_as_float(u * g.up), second = __uint_as_float(u & g.high);
    o.v[i] = interleaved ? f2(second, first) : f2(first, second);
  }
  return o;
}
__device__ __forceinline__ Row8 rotated(const Row8& x, const Row8& other, const Angles& g) {
  Row8 y;
#pragma unroll
  for (int i = 0; i < 4; ++i) y.v[i] = fma2(other.v[i], g.cross[i], mul2(x.v[i], g.own[i]));
  return y;
}

// One 8-channel piece of a quantised row: codes of x / scale (scale not a number: code 0, the
// scale itself then marks the row).
__device__ __forceinline__ uint2 e4m3_codes(const Row8& x, float scale) {
  uint32_t w[2] = {0, 0};
  if (scale == scale) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = un2(x.v[i]);
      const __nv_fp8x2_storage_t t =
          __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(v.x, scale), __fdiv_rn(v.y, scale)), __NV_SATFINITE, __NV_E4M3);
      w[i >> 1] |= (uint32_t)t << (16 * (i & 1));
    }
  }
  return make_uint2(w[0], w[1]);
}

// A group of lanes takes `batches` times kRows heads of one token and kind (q, k, v) as an item, one read
// of the token's angles and the weights for all, the next rows' loads under way while it works on these.
// kLoop: more items than groups of a full device; a group then takes several in turn, the next one's
// indexes and first rows under way too (32768 tokens of 96 + 12 heads: 327 us without, 293 with; a few
// tokens, which need neither, 3.7 us with and 3.3 without).
// kAppend: k and v go to the cache, and a negative slot skips its token; else k goes to k_out.
template <int kLanes, bool kAppend, bool kQuant, bool kLoop>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas) norm_rope_kernel(const __grid_constant__ RopeArgs a, int batches) {
  const int lane = threadIdx.x & 31, sub = lane & (kLanes - 1);
  const int rows = kRows * batches;
  const int nq = (a.q.heads + rows - 1) / rows, nk = (a.k.heads + rows - 1) / rows, nv = (a.v.heads + rows - 1) / rows;
  const uint32_t per_token = nq + nk + nv;
  const uint32_t items = (uint32_t)(a.tokens * per_token);  // (below 2^27: checked by the host)
  const int in_step = 2 * a.d;                              // bytes between rows

  // an item: its token, its kind (0 q, 1 k, 2 v) and heads, and what is loaded ahead for it
  struct Item {
    int64_t token;
    const uint8_t* src;
    int kind, head0, left, pos, slot;  // left: rows from here on
  };
  auto heads_of = [&](int kind) { return kind == 0 ? a.q.heads : kind == 1 ? a.k.heads : a.v.heads; };
  auto begin = [&](uint32_t n) {
    Item t;
    const bool on = n < items;
    t.token = on ? n / per_token : 0;
    const int part = (int)(on ? n % per_token : 0);
    t.kind = part < nq ? 0 : part < nq + nk ? 1 : 2;
    t.head0 = (part - (t.kind == 0 ? 0 : t.kind == 1 ? nq : nq + nk)) * rows;
    t.left = on ? min(heads_of(t.kind) - t.head0, rows) : 0;
    const __nv_bfloat16* x = t.kind == 0 ? a.q.x : t.kind == 1 ? a.k.x : a.v.x;
    const int64_t stride = t.kind == 0 ? a.q.stride : t.kind == 1 ? a.k.stride : a.v.stride;
    t.src = reinterpret_cast<const uint8_t*>(x + t.token * stride + (int64_t)t.head0 * a.d + 8 * sub);
    // (the indexes before the rows: loads come back in order, and the angles wait for the position)
    t.slot = kAppend && on ? __ldg(a.slots + t.token) : 0;
    t.pos = on && a.cos_sin ? __ldg(a.positions + t.token) : 0;
    return t;
  };
  const bool dim_on = 8 * sub < a.d;
  auto load_rows = [&](RowVec (&r)[kRows], const uint8_t* src, int left) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) r[i] = load_row(reinterpret_cast<const __nv_bfloat16*>(src + i * in_step), dim_on && i < left);
  };
  constexpr uint32_t kGroups = kRopeThreads / kLanes;
  RowVec raw[kRows], more[kRows];
  Item now = begin(blockIdx.x * kGroups + threadIdx.x / kLanes);
  load_rows(raw, now.src, now.left);
#pragma unroll 1
  for (uint32_t first = blockIdx.x * kGroups; first < items; first += gridDim.x * kGroups) {
    Item after = {};
    if (kLoop) after = begin(first + gridDim.x * kGroups + threadIdx.x / kLanes);
    const int64_t token = now.token;
    const int kind = now.kind, head0 = now.head0, pos = now.pos;
    int left = now.left, slot = now.slot;
    const uint8_t* src = now.src;
    bool live = left > 0;  // (every lane stays for the shuffles)
    const int heads = heads_of(kind);
    const float* weight = kind == 0 ? a.q.w : kind == 1 ? a.k.w : nullptr;
    // (the turns of the warp's group with the most: every lane takes part in every exchange)
    int turns = (left + kRows - 1) / kRows;
    turns = max(turns, __shfl_xor_sync(0xffffffffu, turns, 16));
    if (kLanes == 8) turns = max(turns, __shfl_xor_sync(0xffffffffu, turns, 8));
    if (kAppend && live) {
      if (slot >= a.num_slots) {
        if (a.status) atomicOr(a.status, kStatusBadIndex);
        slot = -1;
      }
      live = slot >= 0;
    }
    const float* angles_row = nullptr;
    if (live && a.cos_sin) {
      if (pos < 0 || pos >= a.max_pos) {
        if (a.status) atomicOr(a.status, kStatusBadIndex);
        live = false;
      } else {
        angles_row = a.cos_sin + (int64_t)pos * a.rot;
      }
    }
    const bool norm = weight != nullptr;
    Angles ang;
    load_angles<kLanes, false>(ang, kind == 2 ? nullptr : angles_row, a.rot, a.interleaved, weight, dim_on);

    // where the rows go, and the bytes between them
    const bool to_cache = kAppend && kind != 0;
    uint8_t* dst;
    float* scale_at = nullptr;
    int out_step = in_step;
    if (!to_cache) {
      __nv_bfloat16* out = kind == 0 ? a.q_out : a.k_out;
      dst = reinterpret_cast<uint8_t*>(out + (token * heads + head0) * a.d + 8 * sub);
    } else {
      constexpr int kBytes = kQuant ? 1 : 2;
      const int64_t page = slot >> a.page_shift;
      const int64_t line = ((int64_t)head0 << a.page_shift) + (slot & ((1 << a.page_shift) - 1));
      const int64_t at = page * (kind == 1 ? a.k_page_stride : a.v_page_stride) + line * a.d + 8 * sub;
      dst = static_cast<uint8_t*>(kind == 1 ? a.k_cache : a.v_cache) + at * kBytes;
      out_step = (a.d * kBytes) << a.page_shift;
      if (kQuant) scale_at = (kind == 1 ? a.k_scale : a.v_scale) + ((page * heads) << a.page_shift) + line;
    }
    const float inv_d = 1.f / (float)a.d;
    const bool write = live && dim_on;

    auto work = [&](const RowVec (&cur)[kRows], RowVec (&next)[kRows], bool last) {
      load_rows(next, last ? after.src : src + kRows * in_step, last ? after.left : left - kRows);
      float ss[kRows];
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const Row8 x = to_float(cur[i]);
        F2 t = mul2(x.v[0], x.v[0]);
#pragma unroll
        for (int j = 1; j < 4; ++j) t = fma2(x.v[j], x.v[j], t);
        const float2 u = un2(t);
        ss[i] = u.x + u.y;
      }
      const float total = sum4<kLanes>(ss);
      const float rr = norm ? rsqrtf(total * inv_d + a.eps) : 1.f;
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const float r = __shfl_sync(0xffffffffu, rr, sum4_lane<kLanes>(i));
        Row8 x = rotated(to_float(cur[i]), paired(cur[i], ang, a.interleaved), ang);
        const F2 r2 = f2(r, r);
#pragma unroll
        for (int j = 0; j < 4; ++j) x.v[j] = mul2(x.v[j], r2);
        const bool on = write && i < left;
        uint32_t big = 0;
        if (kQuant) {
          // the largest magnitude by its bits: an infinity or NaN is larger than every number
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 t = un2(x.v[j]);
            big = max(big, max(__float_as_uint(t.x) & 0x7fffffffu, __float_as_uint(t.y) & 0x7fffffffu));
          }
          big = group_max<kLanes>(big);
        }
        if (!on) continue;
        if (kQuant && to_cache) {
          const float scale = big >= 0x7f800000u ? __uint_as_float(0x7fffffffu) : fmaxf(__fdiv_rn(__uint_as_float(big), kE4M3Max), kKvScaleFloor);
          *reinterpret_cast<uint2*>(dst + i * out_step) = e4m3_codes(x, scale);
          if (sub == 0) scale_at[i << a.page_shift] = scale;
        } else {
          // (values go to a bf16 cache as they are)
          *reinterpret_cast<uint4*>(dst + i * out_step) =
              kAppend && !kQuant && kind == 2 ? make_uint4(cur[i].u[0], cur[i].u[1], cur[i].u[2], cur[i].u[3]) : to_bf16(x);
        }
      }
      left -= kRows;
      src += kRows * in_step;
      dst += kRows * out_step;
      if (kQuant) scale_at += (int64_t)kRows << a.page_shift;
    };
#pragma unroll 1
    for (int turn = 0; turn < turns; turn += 2) {
      work(raw, more, turn + 1 >= turns);
      if (turn + 1 < turns) {
        work(more, raw, turn + 2 >= turns);
      } else if (kLoop) {
#pragma unroll
        for (int i = 0; i < kRows; ++i) raw[i] = more[i];
      }
    }
    if (!kLoop) break;
    now = after;
  }
}

// The gradient.  y = rotation(x r w): g = rotation^T dy, dw_c = sum over rows of g_c x_c r,
// u = g w, dx = r (u - x r^2 mean_c(u_c x_c)); without a norm dx = g.  A persistent grid: each lane
// keeps its channels' sums of dw over all its rows; they meet once per block, and the blocks'
// partial sums in a second launch, in a fixed order (no atomics).  A group takes up to kBwdTurns
// times two rows of one token, the next two under way while it works on these (and of its next token,
// with the position: 4096 tokens of 96 + 12 heads 69 us, without 71).
constexpr int kBwdTurns = 8;

template <int kLanes>
__global__ void __launch_bounds__(kThreads, 2) norm_rope_bwd_kernel(const __grid_constant__ RopeBwdArgs a, int most_turns, int q_blocks) {
  constexpr int kGroups = kThreads / kLanes;
  const int lane = threadIdx.x & 31, sub = lane & (kLanes - 1), group = threadIdx.x / kLanes;
  const bool lane_on0 = 8 * sub < a.d;
  __shared__ __align__(16) float s_w[kGroups][kAttnMaxDim];
  sm100::griddep_launch_dependents();
  const bool kind = blockIdx.x >= q_blocks;  // queries, or keys
  const uint32_t block = kind ? blockIdx.x - q_blocks : blockIdx.x, blocks = kind ? gridDim.x - q_blocks : q_blocks;
  const HeadRows in = kind ? a.k : a.q;
  const __nv_bfloat16* dy = kind ? a.dyk : a.dyq;
  __nv_bfloat16* dx = kind ? a.dk : a.dq;
  const int turns = min(most_turns, (in.heads + 1) / 2);
  const int parts = (in.heads + 2 * turns - 1) / (2 * max(turns, 1));
  const int items = (int)(a.tokens * parts);  // (below 2^31: checked by the host)
  const bool norm = in.w != nullptr;
  const float inv_d = 1.f / (float)a.d;
  F2 w[4], dw[4];
  {
    float w8[8];
    load8(in.w + 8 * sub, w8, norm && lane_on0, 1.f);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      w[j] = f2(w8[2 * j], w8[2 * j + 1]);
      dw[j] = f2(0.f, 0.f);
    }
  }
  // an item: two rows at a time of one token; its position and first rows are loaded ahead
  RowVec rx[2], rg[2];
  auto load_two = [&](int64_t token, int head, bool on) {
    const __nv_bfloat16* x_row = in.x + token * in.stride + (int64_t)head * a.d + 8 * sub;
    const __nv_bfloat16* dy_row = dy + (token * in.heads + head) * a.d + 8 * sub;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      rx[i] = load_row(x_row + i * a.d, on && lane_on0 && head + i < in.heads);
      rg[i] = load_row(dy_row + i * a.d, on && lane_on0 && head + i < in.heads);
    }
  };
  uint32_t item = block * kGroups + group;
  int pos = item < (uint32_t)items && a.cos_sin ? __ldg(a.positions + item / (uint32_t)parts) : 0;
  load_two(item / (uint32_t)parts, (int)(item % (uint32_t)parts) * 2 * turns, item < (uint32_t)items);
  // (all of a block's groups run the same number of turns: the shuffles are for whole warps)
  for (uint32_t first = block * kGroups; first < (uint32_t)items; first += blocks * kGroups) {
    const int64_t token = item / (uint32_t)parts;
    bool live = item < (uint32_t)items;
    int head0 = (int)(item % (uint32_t)parts) * 2 * turns;
    item += blocks * kGroups;
    const int64_t next_token = item / (uint32_t)parts;
    const int next_head = (int)(item % (uint32_t)parts) * 2 * turns;
    const bool next_on = item < (uint32_t)items;
    const int next_pos = next_on && a.cos_sin ? __ldg(a.positions + next_token) : 0;
    const bool here = live;
    const float* row = nullptr;
    if (live && a.cos_sin) {
      if (pos < 0 || pos >= a.max_pos) {
        if (a.status) atomicOr(a.status, kStatusBadIndex);
        live = false;
      } else {
        row = a.cos_sin + (int64_t)pos * a.rot;
      }
    }
    Angles ang;
    load_angles<kLanes, true>(ang, row, a.rot, a.interleaved, nullptr, lane_on0);
#pragma unroll 1
    for (int turn = 0; turn < turns; ++turn, head0 += 2) {
      const RowVec cx[2] = {rx[0], rx[1]}, cg[2] = {rg[0], rg[1]};
      if (turn + 1 < turns) load_two(token, head0 + 2, here);
      else load_two(next_token, next_head, next_on);
      Row8 g[2];
      float sums[4];  // of x^2 and of u x, both rows
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        g[i] = rotated(to_float(cg[i]), paired(cg[i], ang, a.interleaved), ang);
        const Row8 x = to_float(cx[i]);
        F2 ss = f2(0.f, 0.f), ux = f2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          ss = fma2(x.v[j], x.v[j], ss);
          ux = fma2(mul2(g[i].v[j], w[j]), x.v[j], ux);
        }
        const float2 s2 = un2(ss), u2 = un2(ux);
        sums[i] = s2.x + s2.y;
        sums[2 + i] = u2.x + u2.y;
      }
      const float total = sum4<kLanes>(sums);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float ss = __shfl_sync(0xffffffffu, total, sum4_lane<kLanes>(i));
        const float ux = __shfl_sync(0xffffffffu, total, sum4_lane<kLanes>(2 + i));
        Row8 out = g[i];
        if (norm) {
          const float r = rsqrtf(ss * inv_d + a.eps);
          const float k = -(ux * inv_d * r * r * r);
          const F2 r2 = f2(r, r), k2 = f2(k, k);
          const Row8 x = to_float(cx[i]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            // (a skipped token adds nothing, nor does a place behind the last head: r is infinite there where eps is 0)
            if (live && head0 + i < in.heads) dw[j] = fma2(mul2(g[i].v[j], r2), x.v[j], dw[j]);
            out.v[j] = fma2(x.v[j], k2, mul2(mul2(g[i].v[j], w[j]), r2));
          }
        }
        if (here && lane_on0 && head0 + i < in.heads)  // (a skipped token: zeros)
          *reinterpret_cast<uint4*>(dx + (token * in.heads + head0 + i) * a.d + 8 * sub) = live ? to_bf16(out) : make_uint4(0, 0, 0, 0);
      }
    }
    pos = next_pos;
  }
  if (!norm) return;
  __syncthreads();
  if (lane_on0) {
#pragma unroll
    for (int j = 0; j < 4; ++j) *reinterpret_cast<float2*>(&s_w[group][8 * sub + 2 * j]) = un2(dw[j]);
  }
  __syncthreads();
  for (int ch = threadIdx.x; ch < a.d; ch += kThreads) {
    float t = 0.f;
#pragma unroll
    for (int gr = 0; gr < kGroups; ++gr) t += s_w[gr][ch];
    a.partials[(int64_t)blockIdx.x * kAttnMaxDim + ch] = t;
  }
}

// dw = sum over the blocks' partial sums: one block per projection, 8 slices of blocks per channel.
__global__ void __launch_bounds__(1024) norm_rope_dw_kernel(const float* partials, int q_blocks, int blocks, float* dwq, float* dwk, int d) {
  __shared__ float s[8][kAttnMaxDim];
  const int ch = threadIdx.x & 127, slice = threadIdx.x >> 7, kind = blockIdx.x;
  sm100::griddep_wait();
  float t = 0.f;
  if (ch < d) {
#pragma unroll 8
    for (int i = (kind ? q_blocks : 0) + slice; i < (kind ? blocks : q_blocks); i += 8) t += partials[(int64_t)i * kAttnMaxDim + ch];
  }
  s[slice][ch] = t;
  __syncthreads();
  float* out = kind ? dwk : dwq;
  if (slice == 0 && ch < d && out) {
#pragma unroll
    for (int i = 1; i < 8; ++i) t += s[i][ch];
    out[ch] = t;
  }
}

// The rows of the packed outputs from the cache: a group of lanes takes kReadRows of the 2 heads rows (K,
// then V) of one token, or, with one or two heads, those of kPer consecutive tokens.  Bound by HBM: the cache rows read once, the bf16 rows written once.
template <int kLanes, bool kQuant, int kReadRows, int kPer>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const __grid_constant__ KvReadArgs a) {
  constexpr int kGroups = kThreads / kLanes;
  const int sub = threadIdx.x & (kLanes - 1);
  bool bad = false;
  for (int n = threadIdx.x; n < a.num_seqs; n += kThreads) {
    const int64_t b = a.cu_seqlens[n], e = a.cu_seqlens[n + 1];
    bad |= b > e || (n == 0 && b != 0) || e > a.total || e - b > (int64_t)a.max_pages << a.page_shift;
  }
  if (__syncthreads_or(bad)) {  // nothing is written
    if (threadIdx.x == 0 && a.status) atomicOr(a.status, kStatusBadSeqlens);
    return;
  }
  const int64_t total = a.cu_seqlens[a.num_seqs];
  constexpr int kTokenRows = kReadRows / kPer;  // (where kPer > 1 exactly the 2 heads rows of a token: so the host picks kPer)
  const int parts = (2 * a.heads + kTokenRows - 1) / kTokenRows;
  const uint32_t items = (uint32_t)((total + kPer - 1) / kPer * parts);  // (below 2^31: checked by the host)
  if (8 * sub >= a.d) return;
  for (uint32_t item = blockIdx.x * kGroups + threadIdx.x / kLanes; item < items; item += gridDim.x * kGroups) {
    const int64_t row0 = (int64_t)(item / (uint32_t)parts) * kPer;
    const int r0 = (int)(item % (uint32_t)parts) * kTokenRows;
    int lo = 0, hi = a.num_seqs - 1;  // the last sequence that begins at or before the row and is not empty
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (__ldg(a.cu_seqlens + mid) <= row0) lo = mid;
      else hi = mid - 1;
    }
    int pages[kPer], at[kPer];  // page -1: the token is left out
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      pages[u] = -1;
      at[u] = 0;
      if (row0 + u >= total) continue;
      if (u > 0)
        while (__ldg(a.cu_seqlens + lo + 1) <= row0 + u) ++lo;
      const int t = (int)(row0 + u - __ldg(a.cu_seqlens + lo));
      pages[u] = __ldg(a.page_table + (int64_t)lo * a.max_pages + (t >> a.page_shift));
      at[u] = t & ((1 << a.page_shift) - 1);
      if ((uint32_t)pages[u] >= (uint32_t)a.num_pages) {
        if (a.status) atomicOr(a.status, kStatusBadIndex);
        pages[u] = -1;
      }
    }
    if (kPer == 1 && pages[0] < 0) continue;
    uint4 v[kReadRows];
    float sc[kReadRows];
#pragma unroll
    for (int i = 0; i < kReadRows; ++i) {
      const int r = r0 + i % kTokenRows, page = pages[i / kTokenRows];
      if (kPer == 1 && r >= 2 * a.heads) break;
      if (kPer > 1 && page < 0) continue;
      const bool is_v = r >= a.heads;
      const int64_t line = ((int64_t)(is_v ? r - a.heads : r) << a.page_shift) + at[i / kTokenRows];
      const int64_t off = (int64_t)page * (is_v ? a.v_page_stride : a.k_page_stride) + line * a.d + 8 * sub;
      const void* cache = is_v ? a.v_cache : a.k_cache;
      if (kQuant) {
        const uint2 c = __ldcs(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(cache) + off));
        v[i] = make_uint4(c.x, c.y, 0, 0);
        sc[i] = __ldg((is_v ? a.v_scale : a.k_scale) + (((int64_t)page * a.heads) << a.page_shift) + line);
      } else {
        v[i] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(cache) + off));
      }
    }
#pragma unroll
    for (int i = 0; i < kReadRows; ++i) {
      const int r = r0 + i % kTokenRows;
      if (kPer == 1 && r >= 2 * a.heads) break;
      if (kPer > 1 && pages[i / kTokenRows] < 0) continue;
      const bool is_v = r >= a.heads;
      if (kQuant) {
        const uint32_t w[2] = {v[i].x, v[i].y};
        Row8 x;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[j >> 1] >> (16 * (j & 1))), __NV_E4M3);
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
          x.v[j] = f2(f.x * sc[i], f.y * sc[i]);
        }
        v[i] = to_bf16(x);
      }
      __nv_bfloat16* out = (is_v ? a.v_out : a.k_out) + ((row0 + i / kTokenRows) * a.heads + (is_v ? r - a.heads : r)) * a.d + 8 * sub;
      __stcs(reinterpret_cast<uint4*>(out), v[i]);
    }
  }
}

template <int kLanes>
cudaError_t launch_rope(const RopeArgs& a, bool append, cudaStream_t stream) {
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  // As many rows per group as leave the device full, and few turns empty (heads that do
  // not fill their groups): at 32 + 8 + 8 heads 4097 tokens take 29 us with 4 rows and 24 with 8 or 16,
  // 256 tokens (e4m3) 5.7 us with 4 and 7.9 with 8; at 96 + 12 heads 32768 tokens take 399 us with 4 rows,
  // 314 with 8, 293 with 16 or 32.
  auto items = [&](int b) { return rope_items(1, a.q.heads, a.k.heads, a.v.heads, b); };
  auto blocks = [&](int b) { return (a.tokens * items(b) * kLanes + kRopeThreads - 1) / kRopeThreads; };
  int batches = 1;
  while (batches < 8 && blocks(2 * batches) >= kRopeCtas * (int64_t)sms && items(2 * batches) * 2 * batches * 8 <= items(1) * 9) batches *= 2;
  const int64_t all = blocks(batches), resident = (int64_t)kRopeCtas * sms;
  if (all == 0) return cudaSuccess;
  const bool loop = all > resident;
  auto kernel = loop ? (!append ? norm_rope_kernel<kLanes, false, false, true> : a.k_scale ? norm_rope_kernel<kLanes, true, true, true>
                                                                                            : norm_rope_kernel<kLanes, true, false, true>)
                     : (!append ? norm_rope_kernel<kLanes, false, false, false> : a.k_scale ? norm_rope_kernel<kLanes, true, true, false>
                                                                                             : norm_rope_kernel<kLanes, true, false, false>);
  kernel<<<(unsigned)(loop ? resident : all), kRopeThreads, 0, stream>>>(a, batches);
  return cudaGetLastError();
}

constexpr int kBwdMaxBlocks = 1024;

}  // namespace

int64_t rope_items(int64_t tokens, int32_t hq, int32_t hk, int32_t hv, int batches) {
  auto n = [batches](int32_t heads) { return ((int64_t)heads + kRows * batches - 1) / (kRows * batches); };
  return tokens * (n(hq) + n(hk) + n(hv));
}

size_t rope_bwd_workspace_bytes() { return kWorkspaceHeader + (size_t)kBwdMaxBlocks * kAttnMaxDim * sizeof(float); }

cudaError_t launch_qk_norm_rope(const RopeArgs& a, cudaStream_t stream) {
  return a.d <= 64 ? launch_rope<8>(a, false, stream) : launch_rope<16>(a, false, stream);
}

cudaError_t launch_kv_append(const RopeArgs& a, cudaStream_t stream) {
  return a.d <= 64 ? launch_rope<8>(a, true, stream) : launch_rope<16>(a, true, stream);
}

cudaError_t launch_qk_norm_rope_bwd(const RopeBwdArgs& a, cudaStream_t stream) {
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const int lanes = a.d <= 64 ? 8 : 16;
  // Two blocks per SM, shared by queries and keys as their work is; fewer rows per group where there
  // would be too few groups for them.
  auto blocks = [&](int heads, int turns) { return (a.tokens * ((heads + 2 * turns - 1) / (2 * turns)) * lanes + kThreads - 1) / kThreads; };
  int turns = 1;
  while (turns < kBwdTurns && blocks(a.q.heads, 2 * turns) + blocks(a.k.heads, 2 * turns) >= 4 * (int64_t)sms) turns *= 2;
  int64_t q_blocks = blocks(a.q.heads, turns), k_blocks = blocks(a.k.heads, turns);
  const int64_t most = std::min(kBwdMaxBlocks, 2 * sms);
  if (q_blocks + k_blocks > most) {
    auto work = [&](int heads) {  // turns per token, the items' last ones not full
      const int n = std::min(turns, (heads + 1) / 2);
      return n > 0 ? (int64_t)((heads + 2 * n - 1) / (2 * n)) * n : 0;
    };
    const int64_t share = most * work(a.q.heads) / (work(a.q.heads) + work(a.k.heads));
    q_blocks = std::min(q_blocks, std::max<int64_t>(share, q_blocks > 0));
    k_blocks = std::min(k_blocks, most - q_blocks);
    if (k_blocks == 0 && a.k.heads > 0) k_blocks = 1;
  }
  const int64_t grid = q_blocks + k_blocks;
  if (grid > 0) {
    if (lanes == 8) norm_rope_bwd_kernel<8><<<(unsigned)grid, kThreads, 0, stream>>>(a, turns, (int)q_blocks);
    else norm_rope_bwd_kernel<16><<<(unsigned)grid, kThreads, 0, stream>>>(a, turns, (int)q_blocks);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (!a.dwq && !a.dwk) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2);
  cfg.blockDim = dim3(1024);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = grid > 0 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, norm_rope_dw_kernel, (const float*)a.partials, (int)q_blocks, (int)grid, a.dwq, a.dwk, a.d);
}

cudaError_t launch_kv_read(const KvReadArgs& a, cudaStream_t stream) {
  if (a.num_seqs == 0 || a.total == 0) return cudaSuccess;
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const int lanes = a.d <= 64 ? 8 : 16;
  // Eight rows per group; four where eight would leave the device half empty (8 heads of 128, bf16: 500
  // tokens 3.3 us with eight and 3.0 with four, 8000 tokens 10.5 and 11.1; e4m3, 8000: 10.5 and 12.1).
  auto blocks = [&](int rows) { return (a.total * ((2 * a.heads + rows - 1) / rows) * lanes + kThreads - 1) / kThreads; };
  const bool few = blocks(8) < 2 * (int64_t)sms;
  // One or two heads: the eight rows are of four or two tokens, where that leaves the device full (128000
  // tokens of one head of 64: bf16 16.7 us with one token and 12.2 with four, e4m3 17.6 and 13.5).
  const int tokens = a.heads > 2 ? 1 : 4 / a.heads;
  const int per = blocks(8) / tokens < 2 * (int64_t)sms ? 1 : tokens;
  const int64_t grid = std::min<int64_t>((blocks(few ? 4 : 8) + per - 1) / per, 16 * sms);
  auto pick = [&](auto quant) {
    constexpr bool kQuant = decltype(quant)::value;
    auto form = [&](auto l) {
      constexpr int kLanes = decltype(l)::value;
      return few ? kv_read_kernel<kLanes, kQuant, 4, 1> : per == 4 ? kv_read_kernel<kLanes, kQuant, 8, 4>
           : per == 2 ? kv_read_kernel<kLanes, kQuant, 8, 2> : kv_read_kernel<kLanes, kQuant, 8, 1>;
    };
    return lanes == 8 ? form(std::integral_constant<int, 8>()) : form(std::integral_constant<int, 16>());
  };
  (a.k_scale ? pick(std::true_type()) : pick(std::false_type()))<<<(unsigned)grid, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace kda
