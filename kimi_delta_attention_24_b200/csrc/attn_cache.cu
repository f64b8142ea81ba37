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
// per lane, and one read of the token's angles for the four.  Everything is fp32 between the one
// load and the one rounding.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "attn_common.cuh"
#include "kda_device.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 4;  // rows of one token that a group of lanes takes at a time

struct RowVec {
  uint32_t u[4];  // 8 bf16
};

__device__ __forceinline__ RowVec load_row(const __nv_bfloat16* p, bool on) {
  RowVec r;
  // (a plain load: the outputs may be written in place)
  const uint4 t = on ? *reinterpret_cast<const uint4*>(p) : make_uint4(0, 0, 0, 0);
  r.u[0] = t.x; r.u[1] = t.y; r.u[2] = t.z; r.u[3] = t.w;
  return r;
}
__device__ __forceinline__ void to_float(const RowVec& r, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = unpack_bf16(r.u[i]);
    x[2 * i] = t.x;
    x[2 * i + 1] = t.y;
  }
}
__device__ __forceinline__ uint4 to_bf16(const float (&x)[8]) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}
__device__ __forceinline__ void load8(const float* p, float (&x)[8], bool on) {
  const float4 a = on ? __ldg(reinterpret_cast<const float4*>(p)) : make_float4(0, 0, 0, 0);
  const float4 b = on ? __ldg(reinterpret_cast<const float4*>(p) + 1) : make_float4(0, 0, 0, 0);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
template <int kLanes>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <int kLanes>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// The rotation seen by one lane (its 8 channels of a row): whether it takes part, the partner lane
// of the half-split pairs, and the angles.  Interleaved pairs lie inside a lane; cs / sn then hold
// four angles.
struct Angles {
  bool on, second;
  int partner;  // lane of the warp
  float cs[8], sn[8];
};

template <int kLanes>
__device__ __forceinline__ void load_angles(Angles& g, const float* row, int rot, int interleaved) {
  const int lane = threadIdx.x & 31, sub = lane & (kLanes - 1);
  g.on = row != nullptr && 8 * sub < rot;
  g.second = g.on && !interleaved && 8 * sub >= rot / 2;
  g.partner = lane;
  if (!g.on) {
#pragma unroll
    for (int i = 0; i < 8; ++i) g.cs[i] = 1.f, g.sn[i] = 0.f;
    return;
  }
  if (interleaved) {
    const float4 c = __ldg(reinterpret_cast<const float4*>(row + 4 * sub));
    const float4 s = __ldg(reinterpret_cast<const float4*>(row + rot / 2 + 4 * sub));
    g.cs[0] = c.x; g.cs[1] = c.y; g.cs[2] = c.z; g.cs[3] = c.w;
    g.sn[0] = s.x; g.sn[1] = s.y; g.sn[2] = s.z; g.sn[3] = s.w;
  } else {
    const int at = 8 * sub - (g.second ? rot / 2 : 0);
    load8(row + at, g.cs, true);
    load8(row + rot / 2 + at, g.sn, true);
    g.partner = g.second ? lane - rot / 16 : lane + rot / 16;
  }
}

// x rotated by the angles (kBack: by the opposite ones); `other`: the partner lane's values
// (half-split pairs only).
template <bool kBack>
__device__ __forceinline__ void rotate(float (&x)[8], const float (&other)[8], const Angles& g, int interleaved) {
  if (!g.on) return;
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float s = kBack ? -g.sn[i] : g.sn[i];
      const float p = x[2 * i], q = x[2 * i + 1];
      x[2 * i] = p * g.cs[i] - q * s;
      x[2 * i + 1] = q * g.cs[i] + p * s;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float s = kBack != g.second ? -g.sn[i] : g.sn[i];  // first half: - other sin; second: + other sin
      x[i] = x[i] * g.cs[i] - other[i] * s;
    }
  }
}

// One 8-channel piece of a quantised row: codes of x / scale (scale not a number: code 0, the
// scale itself then marks the row).
__device__ __forceinline__ uint2 e4m3_codes(const float (&x)[8], float scale) {
  uint32_t w[2] = {0, 0};
  if (scale == scale) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_fp8x2_storage_t t =
          __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(x[2 * i], scale), __fdiv_rn(x[2 * i + 1], scale)), __NV_SATFINITE, __NV_E4M3);
      w[i >> 1] |= (uint32_t)t << (16 * (i & 1));
    }
  }
  return make_uint2(w[0], w[1]);
}

// kAppend: k and v go to the cache, and a negative slot skips its token; else k goes to k_out.
template <int kLanes, bool kAppend, bool kQuant>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const __grid_constant__ RopeArgs a) {
  const int lane = threadIdx.x & 31, sub = lane & (kLanes - 1);
  const int nq = (a.q.heads + kRows - 1) / kRows, nk = (a.k.heads + kRows - 1) / kRows, nv = (a.v.heads + kRows - 1) / kRows;
  const int per_token = nq + nk + nv;
  const uint32_t item = blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;  // (below 2^31: checked by the host)
  const int64_t token = item / (uint32_t)per_token;
  bool live = token < a.tokens;  // (every lane stays for the shuffles)
  const int part = (int)(item % (uint32_t)per_token);
  const int kind = part < nq ? 0 : part < nq + nk ? 1 : 2;
  const HeadRows& in = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
  const int head0 = (part - (kind == 0 ? 0 : kind == 1 ? nq : nq + nk)) * kRows;
  const bool lane_on = live && 8 * sub < a.d;

  RowVec raw[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const bool on = lane_on && head0 + i < in.heads;
    raw[i] = load_row(in.x + token * in.stride + (int64_t)(head0 + i) * a.d + 8 * sub, on);
  }
  int slot = 0;
  if (kAppend && live) {
    slot = __ldg(a.slots + token);
    if (slot >= a.num_slots) {
      if (a.status) atomicOr(a.status, kStatusBadIndex);
      slot = -1;
    }
    live = slot >= 0;
  }
  const float* angles_row = nullptr;
  if (live && a.cos_sin) {
    const int pos = __ldg(a.positions + token);
    if (pos < 0 || pos >= a.max_pos) {
      if (a.status) atomicOr(a.status, kStatusBadIndex);
      live = false;
    } else {
      angles_row = a.cos_sin + (int64_t)pos * a.rot;
    }
  }
  Angles ang;
  load_angles<kLanes>(ang, kind == 2 ? nullptr : angles_row, a.rot, a.interleaved);
  const bool norm = in.w != nullptr;
  const float inv_d = 1.f / (float)a.d;
  float w[8], wp[8];
  load8(in.w + 8 * sub, w, norm && lane_on);
  load8(in.w + 8 * (ang.partner & (kLanes - 1)), wp, norm && lane_on);

#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    float x[8], y[8];
    to_float(raw[i], x);
    RowVec ro;
#pragma unroll
    for (int j = 0; j < 4; ++j) ro.u[j] = __shfl_sync(0xffffffffu, raw[i].u[j], ang.partner);
    to_float(ro, y);
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
    ss = group_sum<kLanes>(ss);
    if (norm) {
      const float r = rsqrtf(ss * inv_d + a.eps);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        x[j] *= r * w[j];
        y[j] *= r * wp[j];
      }
    }
    rotate<false>(x, y, ang, a.interleaved);
    const int head = head0 + i;
    const bool on = live && lane_on && head < in.heads;
    if (!kAppend || kind == 0) {
      __nv_bfloat16* out = kind == 0 ? a.q_out : a.k_out;
      if (on) *reinterpret_cast<uint4*>(out + (token * in.heads + head) * a.d + 8 * sub) = to_bf16(x);
      if (!kQuant) continue;
    }
    if (kAppend) {
      const int64_t page = slot >> a.page_shift;
      const int at = slot & ((1 << a.page_shift) - 1);
      const int64_t row = ((int64_t)head << a.page_shift) + at;
      const int64_t base = page * (kind == 1 ? a.k_page_stride : a.v_page_stride) + row * a.d + 8 * sub;
      if (!kQuant) {
        if (on) *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(kind == 1 ? a.k_cache : a.v_cache) + base) = to_bf16(x);
      } else {
        // the largest magnitude by its bits: an infinity or NaN is larger than every number
        uint32_t big = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) big = max(big, __float_as_uint(x[j]) & 0x7fffffffu);
        big = group_max<kLanes>(big);
        if (kind == 0) continue;
        const float scale = big >= 0x7f800000u ? __uint_as_float(0x7fffffffu) : fmaxf(__fdiv_rn(__uint_as_float(big), kE4M3Max), kKvScaleFloor);
        if (on) {
          *reinterpret_cast<uint2*>(static_cast<uint8_t*>(kind == 1 ? a.k_cache : a.v_cache) + base) = e4m3_codes(x, scale);
          if (sub == 0) (kind == 1 ? a.k_scale : a.v_scale)[((page * in.heads) << a.page_shift) + row] = scale;
        }
      }
    }
  }
}

// The gradient.  y = rotation(x r w): g = rotation^T dy, dw_c = sum over rows of g_c x_c r,
// u = g w, dx = r (u - x r^2 mean_c(u_c x_c)); without a norm dx = g.  A persistent grid: each lane
// keeps its channels' sums of dw over all its rows; they meet once per block, and the blocks'
// partial sums in a second launch, in a fixed order (no atomics).
template <int kLanes>
__global__ void __launch_bounds__(kThreads, 3) norm_rope_bwd_kernel(const __grid_constant__ RopeBwdArgs a) {
  constexpr int kGroups = kThreads / kLanes;
  const int lane = threadIdx.x & 31, sub = lane & (kLanes - 1), group = threadIdx.x / kLanes;
  const bool lane_on0 = 8 * sub < a.d;
  __shared__ float s_w[kGroups][kAttnMaxDim];
  sm100::griddep_launch_dependents();
  for (int kind = 0; kind < 2; ++kind) {
    const HeadRows& in = kind ? a.k : a.q;
    const __nv_bfloat16* dy = kind ? a.dyk : a.dyq;
    __nv_bfloat16* dx = kind ? a.dk : a.dq;
    const int parts = (in.heads + 1) / 2;
    const int items = (int)(a.tokens * parts);  // (below 2^31: checked by the host)
    const bool norm = in.w != nullptr;
    const float inv_d = 1.f / (float)a.d;
    float w[8], dw[8];
    load8(in.w + 8 * sub, w, norm && lane_on0);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[j] = 0.f;
    // (all of a block's groups run the same number of turns: the shuffles are for whole warps)
    for (uint32_t first = blockIdx.x * kGroups; first < (uint32_t)items; first += gridDim.x * kGroups) {
      const uint32_t item = first + group;
      const int64_t token = item / (uint32_t)parts;
      bool live = item < (uint32_t)items;
      const int head0 = (int)(item % (uint32_t)parts) * 2;
      RowVec rx[2], rg[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const bool on = live && lane_on0 && head0 + i < in.heads;
        rx[i] = load_row(in.x + token * in.stride + (int64_t)(head0 + i) * a.d + 8 * sub, on);
        rg[i] = load_row(dy + (token * in.heads + head0 + i) * a.d + 8 * sub, on);
      }
      const float* row = nullptr;
      if (live && a.cos_sin) {
        const int pos = __ldg(a.positions + token);
        if (pos < 0 || pos >= a.max_pos) {
          if (a.status) atomicOr(a.status, kStatusBadIndex);
          live = false;
        } else {
          row = a.cos_sin + (int64_t)pos * a.rot;
        }
      }
      Angles ang;
      load_angles<kLanes>(ang, row, a.rot, a.interleaved);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const bool on = live && lane_on0 && head0 + i < in.heads;
        float x[8], g[8], go[8];
        to_float(rx[i], x);
        to_float(rg[i], g);
        RowVec ro;
#pragma unroll
        for (int j = 0; j < 4; ++j) ro.u[j] = __shfl_sync(0xffffffffu, rg[i].u[j], ang.partner);
        to_float(ro, go);
        rotate<true>(g, go, ang, a.interleaved);
        float ss = 0.f, ux = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          ss = fmaf(x[j], x[j], ss);
          ux = fmaf(g[j] * w[j], x[j], ux);
        }
        ss = group_sum<kLanes>(ss);
        ux = group_sum<kLanes>(ux);
        if (norm) {
          const float r = rsqrtf(ss * inv_d + a.eps);
          const float k = ux * inv_d * r * r;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (live) dw[j] = fmaf(g[j] * r, x[j], dw[j]);
            g[j] = r * (g[j] * w[j] - x[j] * k);
          }
        }
        if (on) *reinterpret_cast<uint4*>(dx + (token * in.heads + head0 + i) * a.d + 8 * sub) = to_bf16(g);
      }
    }
    if (!norm) continue;
    __syncthreads();
    if (lane_on0) {
#pragma unroll
      for (int j = 0; j < 8; ++j) s_w[group][8 * sub + j] = dw[j];
    }
    __syncthreads();
    for (int ch = threadIdx.x; ch < a.d; ch += kThreads) {
      float t = 0.f;
#pragma unroll
      for (int gr = 0; gr < kGroups; ++gr) t += s_w[gr][ch];
      a.partials[((int64_t)blockIdx.x * 2 + kind) * kAttnMaxDim + ch] = t;
    }
  }
}

// dw = sum over the blocks' partial sums: one block per projection, 8 slices of blocks per channel.
__global__ void __launch_bounds__(1024) norm_rope_dw_kernel(const float* partials, int blocks, float* dwq, float* dwk, int d) {
  __shared__ float s[8][kAttnMaxDim];
  const int ch = threadIdx.x & 127, slice = threadIdx.x >> 7, kind = blockIdx.x;
  sm100::griddep_wait();
  float t = 0.f;
  if (ch < d) {
#pragma unroll 8
    for (int i = slice; i < blocks; i += 8) t += partials[((int64_t)i * 2 + kind) * kAttnMaxDim + ch];
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

// The rows of the packed outputs from the cache: a group of lanes takes four of the 2 heads rows (K,
// then V) of one token.  Bound by HBM: the cache rows read once, the bf16 rows written once.
template <int kLanes, bool kQuant>
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
  const int parts = (2 * a.heads + kRows - 1) / kRows;
  const uint32_t items = (uint32_t)(total * parts);  // (below 2^31: checked by the host)
  for (uint32_t item = blockIdx.x * kGroups + threadIdx.x / kLanes; item < items; item += gridDim.x * kGroups) {
    const int64_t row = item / (uint32_t)parts;
    const int r0 = (int)(item % (uint32_t)parts) * kRows;
    int lo = 0, hi = a.num_seqs - 1;  // the last sequence that begins at or before the row and is not empty
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (__ldg(a.cu_seqlens + mid) <= row) lo = mid;
      else hi = mid - 1;
    }
    const int t = (int)(row - __ldg(a.cu_seqlens + lo));
    const int page = __ldg(a.page_table + (int64_t)lo * a.max_pages + (t >> a.page_shift));
    if ((uint32_t)page >= (uint32_t)a.num_pages) {
      if (a.status) atomicOr(a.status, kStatusBadIndex);
      continue;
    }
    const int at = t & ((1 << a.page_shift) - 1);
    if (8 * sub >= a.d) continue;
    uint4 v[kRows];
    float sc[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int r = r0 + i;
      if (r >= 2 * a.heads) break;
      const bool is_v = r >= a.heads;
      const int64_t line = ((int64_t)(is_v ? r - a.heads : r) << a.page_shift) + at;
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
    for (int i = 0; i < kRows; ++i) {
      const int r = r0 + i;
      if (r >= 2 * a.heads) break;
      const bool is_v = r >= a.heads;
      if (kQuant) {
        const uint32_t w[2] = {v[i].x, v[i].y};
        float x[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[j >> 1] >> (16 * (j & 1))), __NV_E4M3);
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
          x[2 * j] = f.x * sc[i];
          x[2 * j + 1] = f.y * sc[i];
        }
        v[i] = to_bf16(x);
      }
      __nv_bfloat16* out = (is_v ? a.v_out : a.k_out) + (row * a.heads + (is_v ? r - a.heads : r)) * a.d + 8 * sub;
      __stcs(reinterpret_cast<uint4*>(out), v[i]);
    }
  }
}

template <int kLanes>
cudaError_t launch_rope(const RopeArgs& a, bool append, cudaStream_t stream) {
  const int64_t items = rope_items(a.tokens, a.q.heads, a.k.heads, a.v.heads);
  if (items == 0) return cudaSuccess;
  const int64_t grid = (items * kLanes + kThreads - 1) / kThreads;
  if (!append) norm_rope_kernel<kLanes, false, false><<<(unsigned)grid, kThreads, 0, stream>>>(a);
  else if (a.k_scale) norm_rope_kernel<kLanes, true, true><<<(unsigned)grid, kThreads, 0, stream>>>(a);
  else norm_rope_kernel<kLanes, true, false><<<(unsigned)grid, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

constexpr int kBwdMaxBlocks = 1024;

}  // namespace

int64_t rope_items(int64_t tokens, int32_t hq, int32_t hk, int32_t hv) {
  auto n = [](int32_t heads) { return ((int64_t)heads + kRows - 1) / kRows; };
  return tokens * (n(hq) + n(hk) + n(hv));
}

size_t rope_bwd_workspace_bytes() { return kWorkspaceHeader + (size_t)kBwdMaxBlocks * 2 * kAttnMaxDim * sizeof(float); }

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
  const int64_t most = a.tokens * ((std::max(a.q.heads, a.k.heads) + 1) / 2);
  int64_t grid = (most * lanes + kThreads - 1) / kThreads;
  grid = std::min<int64_t>(grid, std::min(kBwdMaxBlocks, 6 * sms));
  if (grid > 0) {
    if (lanes == 8) norm_rope_bwd_kernel<8><<<(unsigned)grid, kThreads, 0, stream>>>(a);
    else norm_rope_bwd_kernel<16><<<(unsigned)grid, kThreads, 0, stream>>>(a);
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
  return cudaLaunchKernelEx(&cfg, norm_rope_dw_kernel, (const float*)a.partials, (int)grid, a.dwq, a.dwk, a.d);
}

cudaError_t launch_kv_read(const KvReadArgs& a, cudaStream_t stream) {
  if (a.num_seqs == 0 || a.total == 0) return cudaSuccess;
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const int lanes = a.d <= 64 ? 8 : 16;
  const int64_t items = a.total * ((2 * a.heads + kRows - 1) / kRows);
  const int64_t grid = std::min<int64_t>((items * lanes + kThreads - 1) / kThreads, 8 * sms);
  if (lanes == 8) {
    if (a.k_scale) kv_read_kernel<8, true><<<(unsigned)grid, kThreads, 0, stream>>>(a);
    else kv_read_kernel<8, false><<<(unsigned)grid, kThreads, 0, stream>>>(a);
  } else {
    if (a.k_scale) kv_read_kernel<16, true><<<(unsigned)grid, kThreads, 0, stream>>>(a);
    else kv_read_kernel<16, false><<<(unsigned)grid, kThreads, 0, stream>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace kda
