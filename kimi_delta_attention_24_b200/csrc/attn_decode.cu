// Attention of one or a few new tokens per sequence over the paged key-value cache.
//
// Row r = (new token t, query head) of a sequence and its kv head h sees the keys j of the cache with
// j <= p (p = len - new + t, its own position) and, with a window W, j > p - W:
//     z_j = scale q . K_j,  capped: z = cap tanh(z / cap);   o = sum_j e^{z_j} V_j / sum_j e^{z_j}
// in one pass over K and V with the running maximum m and sum l of the softmax (base 2).
//
// What bounds it: every key and value row is read once and used by G T rows (G query heads per kv
// head, T new tokens), 4 G T flops per 2 x 2 bytes (bf16): HBM, until G T is near 64.  So the design
// is a stream of cache tiles with little else:
//   - Split: the (sequence, kv head, row block) units are laid end to end as blocks of 4 tiles of
//     keys, and every CTA (two per SM) takes an equal share of all blocks, wherever it begins and
//     ends, so ragged lengths cost no balance.  A unit that several CTAs share leaves fp32 partial
//     results (o, m, l) in the workspace, joined in a fixed order by a second, dependent launch.
//   - Each of a CTA's 4 warps streams its own tiles (one per block) through its own ring of stages, with
//     no CTA barrier: 16-byte cp.async copies into swizzled rows (conflict-free matrix loads), kept two
//     tiles ahead also across the ends of units; about 130 KB of copies in flight per SM.  (TMA boxes
//     instead cost the issuing warp 800 to 900 cycles a tile, four boxes each, of 2600 to 3400.)
//   - The warps' results of a unit meet as a chain through shared memory, so that no warp waits for a
//     slower one before it goes on with the next unit.
//   - Up to 16 rows (32 where a unit has more) form one mma.sync m16n8k16 operand; these instructions
//     run far below their rate here (a tile's 48 take ~100 of the ~360 cycles its bytes take).
//   - bf16 cache: P enters the second product as a bf16 pair hi + lo, so its rounding (2^-17) stays
//     below that of the bf16 output.  e4m3 cache: codes are exact in fp16; the key's scale multiplies
//     the score, and the value's enters the exponent, w_j = 2^(z_j + log2 s_j - M) with M the row's
//     reference of that sum (within 2^8 of its maximum), whatever the scales are; times 2^7 it is rounded
//     to fp16 (2^-11 down to 2^-21 of 2^M).  q (bf16) is scaled by a power of two per row to fit fp16.
#include <cuda_fp16.h>

#include "attn_common.cuh"
#include "kda_device.cuh"

namespace kda {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kCtasPerSm = 2;
constexpr int kMaxCtas = kCtasPerSm * 160;  // bound used for the workspace (148 SMs on a B200)
constexpr float kLazy = 8.0f;         // how far (base 2) a score passes a row's reference before it moves
constexpr float kWeightShift = 7.0f;  // fp16 weights: up to 2^(kLazy + kWeightShift) = 2^15

struct DecodeParams {
  AttnDecodeArgs a;
  int32_t group, rows, row_blocks;  // rows = new_tokens * group, of one (sequence, kv head)
  float* part_o;                    // [2 * CTAs][rows per block][d]
  float2* part_ml;                  // [2 * CTAs][rows per block]
  int4* meta;                       // [CTAs]: first partial, partials, unit, 0
  uint32_t* status;
};

__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// `bytes` (16 or 0) from src, the rest of the 16 zero.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <bool kHalf>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (kHalf)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Four e4m3 codes as two fp16 pairs.
__device__ __forceinline__ void e4m3x4_to_half2(uint32_t four, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(four));
}
__device__ __forceinline__ uint32_t pack_half(float a, float b) {
  __half2 t = __floats2half2_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&t);
}
__device__ __forceinline__ float lg2_approx(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// tanh to about 2 units in the last place: below 1 Lambert's continued fraction cut after its fifth
// denominator, x (945 + 105 x^2 + x^4) / (945 + 420 x^2 + 15 x^4) (off by 6e-8 at 1), above by 1 - 2 / (e^2x + 1).
__device__ __forceinline__ float tanh_fast(float x) {
  const float q = x * x;
  const float near = x * fmaf(q, q + 105.f, 945.f) * rcp_approx(fmaf(q, fmaf(q, 15.f, 420.f), 945.f));
  const float far = fmaf(-2.f, rcp_approx(ex2_approx(x * (2.f * kLog2e)) + 1.f), 1.f);
  return q < 1.f ? near : far;
}

// Tile geometry.  kDP: the head size padded to 64 or 128 channels (the padding is zero in q and in
// the loaded rows); kTok: keys of one warp's tile, 8 KB of K and V together (4 KB for 64 e4m3
// channels); a block is one tile per warp.
template <bool kFp8, int kDP, int kMT>
struct Geo {
  static constexpr int kTok = kFp8 ? 32 : (kDP == 128 ? 16 : 32);
  static constexpr int kRowBytes = kFp8 ? kDP : 128;               // bytes of a row in one column block
  static constexpr int kColBlocks = kFp8 ? 1 : kDP / 64;           // 128-byte column blocks (bf16)
  static constexpr int kOpBytes = kTok * kRowBytes * kColBlocks;   // K (or V) of one tile
  static constexpr int kStageBytes = 2 * kOpBytes;
  static constexpr int kWarpBytes = 16384;
  static constexpr int kStages = kWarpBytes / kStageBytes;
  static constexpr int kBlockTok = kTok * kWarps;
  static constexpr int kScaleBytes = kFp8 ? 3 * kTok * 4 : 0;            // k scales; v scales, then their logarithms; reciprocals
};

// Byte offset of 16-byte chunk `chunk` of row `row` in a swizzled block of kRowBytes-wide rows.
template <int kRowBytes>
__device__ __forceinline__ uint32_t swz(uint32_t row, uint32_t chunk) {
  return kRowBytes == 128 ? row * 128 + ((chunk ^ (row & 7)) << 4) : row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4);
}

// Keys [lo, hi) that any row of a sequence sees.
__device__ __forceinline__ void key_range(const AttnDecodeArgs& a, int b, int& lo, int& hi, uint32_t* status) {
  int len = a.seq_lens[b];
  const int64_t cap = (int64_t)a.max_pages << a.page_shift;
  if (len < 0 || len > cap) {
    if (status) atomicOr(status, kStatusBadIndex);
    len = len < 0 ? 0 : (int)cap;
  }
  hi = len;
  const int64_t first = a.window > 0 ? (int64_t)len - a.new_tokens - a.window + 1 : 0;
  lo = first > 0 ? (int)first : 0;
}

// Blocks of one unit of the sequence; an empty one counts one block (its output still has to be written).
template <int kBlockTok>
__device__ __forceinline__ int num_blocks(int lo, int hi) {
  const int n = (hi + kBlockTok - 1) / kBlockTok - lo / kBlockTok;
  return n > 0 ? n : 1;
}

// What a unit costs beyond its blocks (queries in, the pipeline filled and drained, the warps' results
// joined and written), in blocks: the shares of the CTAs are equal in blocks + kUnitCost per unit.
constexpr int kUnitCost = 3;

// A CTA's share of all units' blocks, piece by piece: next() steps to the blocks [blk, blk + take) of
// the next unit, until the share is used up.
template <int kBlockTok>
struct Walk {
  int64_t left, off;  // cost left in the share; position of its cursor in sequence next_b
  int next_b;
  int b, u, lo, len, n_blk, blk, take;  // the piece
  __device__ __forceinline__ bool next(const AttnDecodeArgs& a, int64_t units_per_seq) {
    while (left > 0) {
      b = next_b;
      key_range(a, b, lo, len, nullptr);
      n_blk = num_blocks<kBlockTok>(lo, len);
      const int n_cost = n_blk + kUnitCost;
      u = (int)(off / n_cost);
      blk = (int)(off - (int64_t)u * n_cost);
      const int step = (int)min((int64_t)(n_cost - blk), left);  // of the unit's cost; its blocks come first
      take = min(n_blk - blk, step);
      left -= step;
      off += step;
      if (off == n_cost * units_per_seq) {
        ++next_b;
        off = 0;
      }
      if (take > 0) return true;
    }
    return false;
  }
  // a warp's tiles of the piece: the first key of tile i is tok0 + i * kBlockTok, i in [i_begin, i_end)
  // (tiles without a key in [lo, len) are left out)
  __device__ __forceinline__ void tiles(int warp, int tile_tok, int& tok0, int& i_begin, int& i_end) const {
    tok0 = (lo / kBlockTok + blk) * kBlockTok + warp * tile_tok;
    i_end = len > tok0 ? min(take, (len - tok0 - 1) / kBlockTok + 1) : 0;
    i_begin = min(i_end, tok0 + tile_tok <= lo ? 1 : 0);
  }
};

template <bool kFp8, int kDP, int kMT>
struct Smem {
  using G = Geo<kFp8, kDP, kMT>;
  static constexpr int kRows = 16 * kMT;
  static constexpr int kQFragBytes = kMT > 1 ? kMT * (kDP / 16) * 32 * 16 : 0;  // one unit's queries
  static constexpr int kStageOff = 0;
  static constexpr int kWarpBytes = G::kWarpBytes;
  static constexpr int kScaleOff = kWarps * kWarpBytes;
  static constexpr int kQOff = kScaleOff + kWarps * G::kStages * G::kScaleBytes;
  static constexpr int kQRowBytes = kMT == 1 ? kRows * kDP * 2 : 0;             // one unit's queries as they are
  static constexpr int kSumOff = kQOff + 2 * kQFragBytes + 3 * kQRowBytes;      // the warps' sum: [kRows x kDP] floats,
  static constexpr int kMlOff = kSumOff + kRows * kDP * 4;               // and each row's maximum and sum
  static constexpr int kScanOff = kMlOff + kMT * 4 * 32 * 4;             // one int64 per warp
  static constexpr int kTotal = kScanOff + 8 * kWarps;
};

template <bool kFp8, int kDP, int kMT>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) attn_decode_kernel(const __grid_constant__ DecodeParams p) {
  using G = Geo<kFp8, kDP, kMT>;
  using SM = Smem<kFp8, kDP, kMT>;
  constexpr int kTok = G::kTok, kNT = kTok / 8, kKS = kDP / 16, kDT = kDP / 8, kRows = SM::kRows;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (sm100::smem_u32(smem_raw) & 1023)) & 1023);
  const AttnDecodeArgs& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  uint8_t* stages = smem + SM::kStageOff + warp * SM::kWarpBytes;
  float* scales = reinterpret_cast<float*>(smem + SM::kScaleOff) + warp * G::kStages * (G::kScaleBytes / 4);
  float4* s_sum = reinterpret_cast<float4*>(smem + SM::kSumOff) + lane;
  float4* s_ml = reinterpret_cast<float4*>(smem + SM::kMlOff) + lane;
  __shared__ int s_any;
  int64_t* s_scan = reinterpret_cast<int64_t*>(smem + SM::kScanOff);
  __shared__ int s_b;
  __shared__ int64_t s_off;

  sm100::griddep_launch_dependents();

  // ---- this CTA's share [w0, w1) of all blocks, and the sequence it begins in
  const int64_t units_per_seq = (int64_t)a.hkv * p.row_blocks;
  const int per = (a.batch + kThreads - 1) / kThreads;
  const int b_first = tid * per, b_last = min(a.batch, b_first + per);
  int64_t mine = 0;
  for (int b = b_first; b < b_last; ++b) {
    int lo, hi;
    key_range(a, b, lo, hi, blockIdx.x == 0 ? p.status : nullptr);
    mine += (num_blocks<G::kBlockTok>(lo, hi) + kUnitCost) * units_per_seq;
  }
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += t;
  }
  if (lane == 31) s_scan[warp] = incl;
  __syncthreads();
  int64_t before = incl - mine, total = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += s_scan[w];
    total += s_scan[w];
  }
  const int64_t ctas = total < (int64_t)gridDim.x ? total : (int64_t)gridDim.x;
  const int64_t cta = blockIdx.x;
  if (cta >= ctas) {
    if (tid == 0) p.meta[cta] = make_int4(0, 0, 0, 0);
    return;
  }
  const int64_t w0 = cta * total / ctas, w1 = (cta + 1) * total / ctas;
  if (mine > 0 && before <= w0 && w0 < before + mine) {
    int64_t at = before;
    for (int b = b_first; b < b_last; ++b) {
      int lo, hi;
      key_range(a, b, lo, hi, nullptr);
      const int64_t n = (num_blocks<G::kBlockTok>(lo, hi) + kUnitCost) * units_per_seq;
      if (w0 < at + n) {
        s_b = b;
        s_off = w0 - at;
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  Walk<G::kBlockTok> in, out;  // the pieces whose tiles this warp loads next, and computes next
  in.left = w1 - w0;
  in.off = s_off;
  in.next_b = s_b;
  out = in;

  const int page_mask = (1 << a.page_shift) - 1;
  // scores to base 2 (to the cap's units): a positive factor, its sign goes to the queries, so that
  // maxima can be taken before it (a factor of zero: zero queries)
  const float base_scale =
      a.scale == 0.f ? 1.f : fmaxf(fabsf(a.softcap > 0.f ? a.scale / a.softcap : a.scale * kLog2e), 1.17549435e-38f);
  const uint32_t q_sign = a.scale < 0.f ? 0x80008000u : 0u, q_keep = a.scale == 0.f ? 0u : 0xffffffffu;

  // ---- the loading side: a ring of stages, kept full across the units' ends
  constexpr int kChunks = kDP * (kFp8 ? 1 : 2) / 16, kPass = 32 / kChunks;  // 16-byte chunks of a row; rows a pass
  const int ld_ch = lane % kChunks, ld_row = lane / kChunks;
  const int row_bytes = a.d * (kFp8 ? 1 : 2);
  const uint32_t ld_bytes = 16 * ld_ch < row_bytes ? 16 : 0;   // (channels beyond the head size: zero)
  const bool one_page = page_mask + 1 >= kTok;                 // a tile lies in one page
  const uint32_t ring = sm100::smem_u32(stages) + (ld_ch / 8) * (kTok * G::kRowBytes);
  const int64_t k_step = a.k_page_stride * (kFp8 ? 1 : 2), v_step = a.v_page_stride * (kFp8 ? 1 : 2);
  const uint8_t* k_base = static_cast<const uint8_t*>(a.k_cache) + (ld_bytes ? 16 * ld_ch : 0);
  const uint8_t* v_base = static_cast<const uint8_t*>(a.v_cache) + (ld_bytes ? 16 * ld_ch : 0);
  int stage_in = 0, stage_out = 0;
  int in_tok = 0, in_i = 0, in_end = 0, in_h = 0, page_next = 0;
  int in_piece = -1, in_slot = 2, ahead = 0;  // the piece being loaded, its place for queries; tiles under way
  bool in_more = true, in_first = false;
  // to the next tile; this lane's page is that of the key it stands for (of the nearest key in [lo, len))
  auto advance = [&]() {
    ++in_i;
    while (in_i >= in_end) {
      in_more = in.next(a, units_per_seq);
      if (!in_more) return;
      ++in_piece;
      in_slot = in_slot == 2 ? 0 : in_slot + 1;
      in_first = true;
      in_h = in.u / p.row_blocks;
      in.tiles(warp, kTok, in_tok, in_i, in_end);
    }
    int tok = in_tok + in_i * G::kBlockTok + (lane & (kTok - 1));
    tok = tok < in.lo ? in.lo : (tok >= in.len ? in.len - 1 : tok);
    page_next = a.page_table[(int64_t)in.b * a.max_pages + (tok >> a.page_shift)];
  };
  // the copies of the next tile, as one group
  auto issue = [&]() {
    {
      int page = page_next;
      if ((uint32_t)page >= (uint32_t)a.num_pages) {  // never read outside the cache
        if (p.status) atomicOr(p.status, kStatusBadIndex);
        page = 0;
      }
      const int t0 = in_tok + in_i * G::kBlockTok;
      const uint32_t st = ring + stage_in * G::kStageBytes;
      if (kMT == 1 && in_first) {
        // the unit's queries come with its first tile: a load that is waited for at the unit's start
        // would queue behind all the copies under way.  All four warps copy them (the same bytes); of
        // three places the one behind a warp that lags and before one that leads is free.
        in_first = false;
        constexpr int kQChunks = kDP * 2 / 16, kQPass = 32 / kQChunks;
        const int base = (in.u - in_h * p.row_blocks) * kRows, ch = lane % kQChunks;
        const int live = min(kRows, p.rows - base);
        const uint32_t dst = sm100::smem_u32(smem + SM::kQOff + in_slot * SM::kQRowBytes);
        for (int r = lane / kQChunks; r < live; r += kQPass) {
          const int t = (base + r) / p.group, head = in_h * p.group + base + r - t * p.group;
          const __nv_bfloat16* src = a.q + (((int64_t)in.b * a.new_tokens + t) * a.hq + head) * a.d;
          const bool on = 8 * ch < a.d;
          cp_async16(dst + r * (kDP * 2) + ((ch ^ (r & 7)) << 4), src + (on ? 8 * ch : 0), on ? 16 : 0);
        }
      }
      auto copy_rows = [&](int i, const uint8_t* ks, const uint8_t* vs) {
        const uint32_t row = i * kPass + ld_row;
        const uint32_t dst = st + swz<G::kRowBytes>(row, ld_ch % (G::kRowBytes / 16));
        cp_async16(dst, ks, ld_bytes);
        cp_async16(dst + G::kOpBytes, vs, ld_bytes);
      };
      if (one_page) {
        const int64_t line = (((int64_t)in_h << a.page_shift) + (t0 & page_mask) + ld_row) * row_bytes;
        const uint8_t* ks = k_base + page * k_step + line;
        const uint8_t* vs = v_base + page * v_step + line;
#pragma unroll
        for (int i = 0; i < kTok / kPass; ++i) {
          copy_rows(i, ks, vs);
          ks += kPass * row_bytes;
          vs += kPass * row_bytes;
        }
      } else {
#pragma unroll 2
        for (int i = 0; i < kTok / kPass; ++i) {
          const int row = i * kPass + ld_row;
          const int pg = __shfl_sync(0xffffffffu, page, row);
          const int64_t line = (((int64_t)in_h << a.page_shift) + ((t0 + row) & page_mask)) * row_bytes;
          copy_rows(i, k_base + pg * k_step + line, v_base + pg * v_step + line);
        }
      }
      if (kFp8) {
        const int64_t s = (((int64_t)page * a.hkv + in_h) << a.page_shift) + ((t0 + lane) & page_mask);
        const uint32_t dst = sm100::smem_u32(scales + stage_in * 3 * kTok + lane);
        cp_async4(dst, a.k_scale + s);
        cp_async4(dst + kTok * 4, a.v_scale + s);
      }
    }
    cp_async_commit();
    if (++stage_in == G::kStages) stage_in = 0;
    ++ahead;
    advance();
  };
  advance();

  int4 meta = make_int4(0, 0, 0, 0);
  int pieces = 0, slot_out = 0;
  bool more = out.next(a, units_per_seq);
  while (more) {
    const int b = out.b, len = out.len, lo = out.lo, blk = out.blk, take = out.take, n_blk = out.n_blk, u = out.u;
    const int h = u / p.row_blocks, row_base = (u - h * p.row_blocks) * kRows;
    int tok0, i_begin, i_end;
    out.tiles(warp, kTok, tok0, i_begin, i_end);
    more = out.next(a, units_per_seq);

    // ---- the rows' key ranges, their queries as fragments
    uint4* q_smem = reinterpret_cast<uint4*>(smem + SM::kQOff + (pieces & 1) * SM::kQFragBytes) + lane;
    uint32_t qf[kMT == 1 ? kKS : 1][4];
    float rscale[kMT][2];   // score factor of rows g and g + 8
    int row_hi[kMT][2], row_lo[kMT][2];
    const __nv_bfloat16* src[kMT][2];
#pragma unroll
    for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int r = row_base + mt * 16 + s * 8 + g;
        const bool ok = r < p.rows;
        const int t = ok ? r / p.group : 0;
        const int head = h * p.group + (ok ? r - t * p.group : 0);
        src[mt][s] = ok ? a.q + (((int64_t)b * a.new_tokens + t) * a.hq + head) * a.d : nullptr;
        const int pos = len - a.new_tokens + t;
        row_hi[mt][s] = ok ? pos + 1 : 0;
        row_lo[mt][s] = a.window > 0 && pos >= a.window ? pos - a.window + 1 : 0;
        rscale[mt][s] = base_scale;
      }
    auto make_fragments = [&]() {
      const uint8_t* q_rows = smem + SM::kQOff + slot_out * SM::kQRowBytes;
      // 8 (4) channels of row tile mt's row 8 s + g
      auto load16 = [&](int mt, int s, int ch) {
        if (kMT == 1) return *reinterpret_cast<const uint4*>(q_rows + (8 * s + g) * (kDP * 2) + (((ch / 8) ^ g) << 4));
        return src[mt][s] && ch < a.d ? __ldg(reinterpret_cast<const uint4*>(src[mt][s] + ch)) : make_uint4(0, 0, 0, 0);
      };
      auto load4 = [&](int mt, int s, int ch) {
        if (kMT == 1) return *reinterpret_cast<const uint32_t*>(q_rows + (8 * s + g) * (kDP * 2) + (((ch / 8) ^ g) << 4) + (ch % 8) * 2);
        return src[mt][s] && ch < a.d ? __ldg(reinterpret_cast<const unsigned int*>(src[mt][s] + ch)) : 0u;
      };
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt) {
        uint32_t f[kKS][4];
        if (!kFp8) {
#pragma unroll
          for (int ks = 0; ks < kKS; ++ks)
#pragma unroll
            for (int j = 0; j < 4; ++j) f[ks][j] = (load4(mt, j & 1, ks * 16 + (j >> 1) * 8 + 2 * c) & q_keep) ^ q_sign;
        } else {
          // channels 64 j + 16 c + 4 s + {0..3} are k-step 4 j + s of this thread (as the key bytes are read)
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            uint32_t wv[kDP / 64][8];
            float big = 0.f;
#pragma unroll
            for (int j = 0; j < kDP / 64; ++j) {
              const uint4 v0 = load16(mt, s, 64 * j + 16 * c), v1 = load16(mt, s, 64 * j + 16 * c + 8);
              wv[j][0] = v0.x; wv[j][1] = v0.y; wv[j][2] = v0.z; wv[j][3] = v0.w;
              wv[j][4] = v1.x; wv[j][5] = v1.y; wv[j][6] = v1.z; wv[j][7] = v1.w;
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                wv[j][i] = (wv[j][i] & q_keep) ^ q_sign;
                const float2 t = unpack_bf16(wv[j][i]);
                big = fmaxf(big, fmaxf(fabsf(t.x), fabsf(t.y)));
              }
            }
            big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
            big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
            // the power of two below the row's largest magnitude (exact factors)
            int e = (int)((__float_as_uint(big) >> 23) & 255) - 127;
            e = big == 0.f || e > 126 ? 0 : (e < -100 ? -100 : e);
            const float down = __uint_as_float((uint32_t)(127 - e) << 23);
            rscale[mt][s] = base_scale * __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
            for (int j = 0; j < kDP / 64; ++j)
#pragma unroll
              for (int q4 = 0; q4 < 4; ++q4) {
                const float2 t0 = unpack_bf16(wv[j][2 * q4]), t1 = unpack_bf16(wv[j][2 * q4 + 1]);
                f[4 * j + q4][s] = pack_half(t0.x * down, t0.y * down);
                f[4 * j + q4][s + 2] = pack_half(t1.x * down, t1.y * down);
              }
          }
        }
        if (kMT == 1) {
#pragma unroll
          for (int ks = 0; ks < kKS; ++ks)
#pragma unroll
            for (int j = 0; j < 4; ++j) qf[kMT == 1 ? ks : 0][j] = f[ks][j];
        } else {
          // all four warps write the same; two units' queries alternate, and a warp is at most one unit
          // ahead of another (the chain of sums below)
#pragma unroll
          for (int ks = 0; ks < kKS; ++ks) q_smem[(mt * kKS + ks) * 32] = make_uint4(f[ks][0], f[ks][1], f[ks][2], f[ks][3]);
        }
      }
      if (kMT > 1) __syncwarp();
    };
    if (kMT > 1) make_fragments();

    float o[kMT][kDT][4];
    float m[kMT][2], l[kMT][2];
#pragma unroll
    for (int mt = 0; mt < kMT; ++mt) {
#pragma unroll
      for (int j = 0; j < kDT; ++j) o[mt][j][0] = o[mt][j][1] = o[mt][j][2] = o[mt][j][3] = 0.f;
      m[mt][0] = m[mt][1] = -INFINITY;
      l[mt][0] = l[mt][1] = 0.f;
    }
    // tiles whose every key every row sees need no mask
    const int all_hi = len - a.new_tokens + 1, all_lo = a.window > 0 ? len - a.window : 0;

    for (int i = i_begin; i < i_end; ++i) {
      // refill the stages that the tiles before have left, at most into the next unit
      while (ahead < G::kStages && in_more && in_piece <= pieces + 1) issue();
      if (ahead == G::kStages) cp_async_wait<G::kStages - 1>();
      else if (ahead == 2) cp_async_wait<1>();
      else if (ahead == 1) cp_async_wait<0>();
      else cp_async_wait<2>();
      __syncwarp();
      if (kMT == 1 && i == i_begin) make_fragments();
      uint8_t* st = stages + stage_out * G::kStageBytes;
      const uint32_t ks_addr = sm100::smem_u32(st), vs_addr = ks_addr + G::kOpBytes;
      float* sc = scales + stage_out * 3 * kTok;
      if (kFp8) {
        // once per key: the logarithm of its value scale and the reciprocal.  (A scale that is not a
        // number makes the rows that see its key so, by way of the logarithm; its reciprocal stays
        // finite, for the rows that do not see it.)
        const float v = sc[kTok + lane];
        sc[kTok + lane] = lg2_approx(v < 0x1p-100f ? 0x1p-100f : v);
        sc[2 * kTok + lane] = rcp_approx(fmaxf(v, 0x1p-100f));
        __syncwarp();
      }
      const int t0 = tok0 + i * G::kBlockTok;
      const bool edge = t0 + kTok > all_hi || t0 < all_lo;

      // ---- S = Q K^T
      float s[kMT][kNT][4];
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) s[mt][nt][0] = s[mt][nt][1] = s[mt][nt][2] = s[mt][nt][3] = 0.f;
      if (!kFp8) {
        constexpr bool kSplit = kNT == 2;
        float s_odd[kMT][kSplit ? kNT : 1][4] = {};
        const uint32_t mrow = ((lane >> 4) << 3) + (lane & 7), mchunk = (lane >> 3) & 1;
#pragma unroll
        for (int ks = 0; ks < kKS; ++ks) {
          uint32_t qa[kMT][4];
#pragma unroll
          for (int mt = 0; mt < kMT; ++mt) {
            if (kMT == 1) {
#pragma unroll
              for (int j = 0; j < 4; ++j) qa[mt][j] = qf[kMT == 1 ? ks : 0][j];
            } else {
              const uint4 t = q_smem[(mt * kKS + ks) * 32];
              qa[mt][0] = t.x; qa[mt][1] = t.y; qa[mt][2] = t.z; qa[mt][3] = t.w;
            }
          }
#pragma unroll
          for (int n2 = 0; n2 < kNT / 2; ++n2) {
            uint32_t kb[4];
            ldsm4(kb, ks_addr + (ks >> 2) * (kTok * 128) + swz<128>(n2 * 16 + mrow, (ks & 3) * 2 + mchunk));
#pragma unroll
            for (int mt = 0; mt < kMT; ++mt) {
              // (one row tile of 16 keys has two sums only: even and odd steps apart, half the chain)
              float (&s0)[4] = kSplit && (ks & 1) ? s_odd[mt][kSplit ? 2 * n2 : 0] : s[mt][2 * n2];
              float (&s1)[4] = kSplit && (ks & 1) ? s_odd[mt][kSplit ? 2 * n2 + 1 : 0] : s[mt][2 * n2 + 1];
              mma16816<false>(s0, qa[mt], kb[0], kb[1]);
              mma16816<false>(s1, qa[mt], kb[2], kb[3]);
            }
          }
        }
        if (kSplit) {
#pragma unroll
          for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) s[mt][nt][e] += s_odd[mt][kSplit ? nt : 0][e];
        }
      } else {
#pragma unroll
        for (int j = 0; j < kDP / 64; ++j) {
          uint32_t qa[kMT][4][4];
#pragma unroll
          for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
            for (int q4 = 0; q4 < 4; ++q4) {
              if (kMT == 1) {
#pragma unroll
                for (int x = 0; x < 4; ++x) qa[mt][q4][x] = qf[kMT == 1 ? 4 * j + q4 : 0][x];
              } else {
                const uint4 t = q_smem[(mt * kKS + 4 * j + q4) * 32];
                qa[mt][q4][0] = t.x; qa[mt][q4][1] = t.y; qa[mt][q4][2] = t.z; qa[mt][q4][3] = t.w;
              }
            }
          uint4 kb[kNT];
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt) kb[nt] = *reinterpret_cast<const uint4*>(st + swz<G::kRowBytes>(nt * 8 + g, 4 * j + c));
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4)
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt) {
              uint32_t b0, b1;
              e4m3x4_to_half2(q4 == 0 ? kb[nt].x : q4 == 1 ? kb[nt].y : q4 == 2 ? kb[nt].z : kb[nt].w, b0, b1);
#pragma unroll
              for (int mt = 0; mt < kMT; ++mt) mma16816<true>(s[mt][nt], qa[mt][q4], b0, b1);
            }
        }
      }

      // ---- scores, masks, the value scales' logarithms.  S becomes z (times the row's factor where it
      // is not yet applied: bf16 without a cap).
      float inv_vs[kFp8 ? kNT : 1][2];
      const bool capped = a.softcap > 0.f;
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) {
        float kf[2] = {1.f, 1.f}, lv[2] = {0.f, 0.f};
        if (kFp8) {
          const float2 k2 = *reinterpret_cast<const float2*>(sc + nt * 8 + 2 * c);
          const float2 l2 = *reinterpret_cast<const float2*>(sc + kTok + nt * 8 + 2 * c);
          const float2 i2 = *reinterpret_cast<const float2*>(sc + 2 * kTok + nt * 8 + 2 * c);
          kf[0] = k2.x;
          kf[1] = k2.y;
          lv[0] = l2.x;
          lv[1] = l2.y;
          inv_vs[kFp8 ? nt : 0][0] = i2.x;
          inv_vs[kFp8 ? nt : 0][1] = i2.y;
        }
        if (capped) {
#pragma unroll
          for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float z = kFp8 ? s[mt][nt][e] * kf[e & 1] : s[mt][nt][e];
              s[mt][nt][e] = fmaf(a.softcap * kLog2e, tanh_fast(z * rscale[mt][e >> 1]), lv[e & 1]);
            }
        } else if (kFp8) {
#pragma unroll
          for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[mt][nt][e] = fmaf(s[mt][nt][e] * kf[e & 1], rscale[mt][e >> 1], lv[e & 1]);
        }
      }
      if (edge) {
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
          for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int j = t0 + nt * 8 + 2 * c + (e & 1);
              if (j >= row_hi[mt][e >> 1] || j < row_lo[mt][e >> 1]) s[mt][nt][e] = -INFINITY;
            }
      }
      // ---- running sum and reference of the exponents; P in place of S.  The reference m of a row is
      // its maximum when it was last moved: it moves (for all rows of the warp) only when a score
      // passes it by kLazy, so P stays below 2^kLazy and most tiles need no exchange between threads.
      bool passed = false;
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float fac = kFp8 || capped ? 1.f : rscale[mt][x];
          float mx = -INFINITY;
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt) mx = fmaxf(mx, fmaxf(s[mt][nt][2 * x], s[mt][nt][2 * x + 1]));
          passed |= mx * fac > m[mt][x] + kLazy;
        }
      if (__any_sync(0xffffffffu, passed)) {
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt) {
          float alpha[2];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float fac = kFp8 || capped ? 1.f : rscale[mt][x];
            float mx = -INFINITY;
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt) mx = fmaxf(mx, fmaxf(s[mt][nt][2 * x], s[mt][nt][2 * x + 1]));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const float mn = fmaxf(m[mt][x], mx * fac);
            alpha[x] = ex2_approx(m[mt][x] - (mn == -INFINITY ? 0.f : mn));
            m[mt][x] = mn;
            l[mt][x] *= alpha[x];
          }
#pragma unroll
          for (int j = 0; j < kDT; ++j) {
            o[mt][j][0] *= alpha[0];
            o[mt][j][1] *= alpha[0];
            o[mt][j][2] *= alpha[1];
            o[mt][j][3] *= alpha[1];
          }
        }
      }
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float fac = kFp8 || capped ? 1.f : rscale[mt][x];
          const float shift = (m[mt][x] == -INFINITY ? 0.f : m[mt][x]) - (kFp8 ? kWeightShift : 0.f);
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float pr = ex2_approx(kFp8 ? s[mt][nt][2 * x + e] - shift : fmaf(s[mt][nt][2 * x + e], fac, -shift));
              s[mt][nt][2 * x + e] = pr;
              l[mt][x] = kFp8 ? fmaf(pr, inv_vs[kFp8 ? nt : 0][e], l[mt][x]) : l[mt][x] + pr;
            }
        }

      if (edge) {
        // Rows of V that no query of the unit sees may hold anything (they may never have been
        // written): zero them, since 0 * inf is not 0.
        constexpr int kRowChunks = G::kColBlocks * G::kRowBytes / 16;
        auto zero_rows = [&](int r0, int r1) {
          for (int x = r0 * kRowChunks + lane; x < r1 * kRowChunks; x += 32) {
            const int r = x / kRowChunks, ch = x % kRowChunks;
            *reinterpret_cast<uint4*>(st + G::kOpBytes + (ch / (G::kRowBytes / 16)) * (kTok * G::kRowBytes) +
                                      swz<G::kRowBytes>(r, ch % (G::kRowBytes / 16))) = make_uint4(0, 0, 0, 0);
          }
        };
        zero_rows(0, lo - t0);
        zero_rows(max(len - t0, 0), kTok);
        if (!kFp8) {
          // Keys that some rows see and others do not: an infinity or NaN in such a row of V must
          // not reach the rows that do not see it.  Take that row out of the product and add it to
          // the rows that see it, element by element.
          const int low_end = min(max(all_lo - t0, 0), kTok);   // keys [lo, all_lo) and [all_hi, len)
          for (int r = max(lo - t0, 0); r < min(len - t0, kTok); ++r) {
            if (r >= low_end && r < all_hi - t0) r = all_hi - t0;
            if (r >= min(len - t0, kTok)) break;
            const int j = t0 + r;
            uint4* at = reinterpret_cast<uint4*>(st + G::kOpBytes + (lane / 8) * (kTok * 128) + swz<128>(r, lane % 8));
            bool odd = false;
            if (lane < kChunks) {
              const uint4 v = *at;
              const uint32_t wv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int x = 0; x < 4; ++x) odd |= (wv[x] & 0x7f80u) == 0x7f80u || (wv[x] & 0x7f800000u) == 0x7f800000u;
            }
            if (!__any_sync(0xffffffffu, odd)) continue;
#pragma unroll
            for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                uint32_t bits = 0;  // P[row][r], held by thread (r % 8) / 2 of the row's four (masks: no local array)
#pragma unroll
                for (int nt = 0; nt < kNT; ++nt) {
                  const uint32_t here = nt == r / 8 ? 0xffffffffu : 0u, second = (r & 1) ? 0xffffffffu : 0u;
                  bits |= here & ((second & __float_as_uint(s[mt][nt][2 * x + 1])) | (~second & __float_as_uint(s[mt][nt][2 * x])));
                }
                const float pr = __uint_as_float(__shfl_sync(0xffffffffu, bits, (lane & ~3) | ((r & 7) >> 1)));
                if (j < row_hi[mt][x] && j >= row_lo[mt][x]) {
#pragma unroll
                  for (int dt = 0; dt < kDT; ++dt) {
                    const float2 v = unpack_bf16(*reinterpret_cast<const uint32_t*>(
                        st + G::kOpBytes + (dt / 8) * (kTok * 128) + swz<128>(r, dt % 8) + 4 * c));
                    o[mt][dt][2 * x] = fmaf(pr, v.x, o[mt][dt][2 * x]);
                    o[mt][dt][2 * x + 1] = fmaf(pr, v.y, o[mt][dt][2 * x + 1]);
                  }
                }
              }
            __syncwarp();
            if (lane < kChunks) *at = make_uint4(0, 0, 0, 0);
          }
        }
        __syncwarp();
      }

      // ---- O += P V
      if (!kFp8) {
        const uint32_t vrow = lane & 15, vchunk = lane >> 4;
#pragma unroll
        for (int kt = 0; kt < kTok / 16; ++kt) {
          uint32_t hi[kMT][4], lo2[kMT][4];
#pragma unroll
          for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
            for (int x = 0; x < 4; ++x)
              split2(s[mt][2 * kt + (x >> 1)][2 * (x & 1)], s[mt][2 * kt + (x >> 1)][2 * (x & 1) + 1], hi[mt][x], lo2[mt][x]);
          // (four loads, then their products, hi before lo: a sum is met again after eight others)
#pragma unroll
          for (int d8 = 0; d8 < kDT / 8; ++d8) {
            uint32_t vb[4][4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int d2 = 4 * d8 + q;
              ldsm4t(vb[q], vs_addr + (d2 >> 2) * (kTok * 128) + swz<128>(kt * 16 + vrow, (d2 & 3) * 2 + vchunk));
            }
#pragma unroll
            for (int part = 0; part < 2; ++part)
#pragma unroll
              for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int mt = 0; mt < kMT; ++mt) {
                  const uint32_t (&pa)[4] = part ? lo2[mt] : hi[mt];
                  mma16816<false>(o[mt][8 * d8 + 2 * q], pa, vb[q][0], vb[q][1]);
                  mma16816<false>(o[mt][8 * d8 + 2 * q + 1], pa, vb[q][2], vb[q][3]);
                }
          }
        }
      } else {
        // column g of product tile j stands for channel (kDP / 8) g + j: a thread's bytes of a row are contiguous
        const uint8_t* vst = st + G::kOpBytes;
#pragma unroll
        for (int kt = 0; kt < kTok / 16; ++kt) {
          uint32_t pa[kMT][4];
#pragma unroll
          for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
            for (int x = 0; x < 4; ++x)
              pa[mt][x] = pack_half(s[mt][2 * kt + (x >> 1)][2 * (x & 1)], s[mt][2 * kt + (x >> 1)][2 * (x & 1) + 1]);
          constexpr int kWords = kDP / 32;  // 32-bit words of a row per thread: 4 or 2
          uint32_t vw[4][kWords];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int r = kt * 16 + (x >> 1) * 8 + 2 * c + (x & 1);
            if (kDP == 128) {
              const uint4 t = *reinterpret_cast<const uint4*>(vst + swz<G::kRowBytes>(r, g));
              vw[x][0] = t.x; vw[x][1] = t.y; vw[x][kWords - 2] = t.z; vw[x][kWords - 1] = t.w;
            } else {
              const uint2 t = *reinterpret_cast<const uint2*>(vst + swz<G::kRowBytes>(r, g >> 1) + 8 * (g & 1));
              vw[x][0] = t.x; vw[x][1] = t.y;
            }
          }
#pragma unroll
          for (int x = 0; x < kWords; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const uint32_t e0 = __byte_perm(vw[0][x], vw[1][x], y ? 0x7362 : 0x5140);
              const uint32_t e1 = __byte_perm(vw[2][x], vw[3][x], y ? 0x7362 : 0x5140);
              uint32_t b00, b01, b10, b11;
              e4m3x4_to_half2(e0, b00, b01);
              e4m3x4_to_half2(e1, b10, b11);
#pragma unroll
              for (int mt = 0; mt < kMT; ++mt) {
                mma16816<true>(o[mt][4 * x + 2 * y], pa[mt], b00, b10);
                mma16816<true>(o[mt][4 * x + 2 * y + 1], pa[mt], b01, b11);
              }
            }
        }
      }
      __syncwarp();  // the stage has been read
      --ahead;
      if (++stage_out == G::kStages) stage_out = 0;
    }

    // ---- the warps' results together, as a chain: each warp adds its own to the sum that the warp
    // before it left in shared memory, and the last one writes the result.  A warp that has passed its
    // sum on goes on with the next unit, whose tiles are under way already.  Barrier w passes the sum
    // from warp w - 1 to warp w; barrier kWarps gives its place back to warp 0.
    // (a row's four threads hold parts of its sum l)
#pragma unroll
    for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        l[mt][x] += __shfl_xor_sync(0xffffffffu, l[mt][x], 1);
        l[mt][x] += __shfl_xor_sync(0xffffffffu, l[mt][x], 2);
      }
    if (warp > 0) sm100::named_bar(warp, 64);
    else if (pieces > 0) sm100::named_bar(kWarps, 64);
    const bool mine_any = i_begin < i_end, sum_any = warp > 0 && s_any;
    if (sum_any) {
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt) {
        const float4 ml = s_ml[mt * 32];
        float f[2], fs[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float mo = x ? ml.z : ml.x, lo2 = x ? ml.w : ml.y;
          const float top = fmaxf(m[mt][x], mo);
          // (a maximum of -inf: no key, or no number; what is added is then 0 or not a number)
          f[x] = m[mt][x] == -INFINITY ? 1.f : ex2_approx(m[mt][x] - top);
          fs[x] = mo == -INFINITY ? 1.f : ex2_approx(mo - top);
          m[mt][x] = top;
          l[mt][x] = l[mt][x] * f[x] + lo2 * fs[x];
        }
#pragma unroll
        for (int j = 0; j < kDT; ++j) {
          const float4 t = s_sum[(mt * kDT + j) * 32];
          o[mt][j][0] = o[mt][j][0] * f[0] + t.x * fs[0];
          o[mt][j][1] = o[mt][j][1] * f[0] + t.y * fs[0];
          o[mt][j][2] = o[mt][j][2] * f[1] + t.z * fs[1];
          o[mt][j][3] = o[mt][j][3] * f[1] + t.w * fs[1];
        }
      }
    }
    __syncwarp();  // the sum has been read
    if (warp < kWarps - 1) {
      if (mine_any || warp == 0) {
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt) {
          s_ml[mt * 32] = make_float4(m[mt][0], l[mt][0], m[mt][1], l[mt][1]);
#pragma unroll
          for (int j = 0; j < kDT; ++j) s_sum[(mt * kDT + j) * 32] = make_float4(o[mt][j][0], o[mt][j][1], o[mt][j][2], o[mt][j][3]);
        }
        if (lane == 0) s_any = mine_any || sum_any;
      }
      __syncwarp();
      sm100::named_bar_arrive(warp + 1, 64);
    } else {
      if (more) sm100::named_bar_arrive(kWarps, 64);
      const bool whole = blk == 0 && take == n_blk;
      const int64_t slot = 2 * cta + (pieces == 0 ? 0 : 1);
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int r = mt * 16 + x * 8 + g, row = row_base + r;
          if (row >= p.rows) continue;
          const float top = m[mt][x], sum = l[mt][x];
          const int t = row / p.group, head = h * p.group + row - t * p.group;
          const int64_t at = ((int64_t)b * a.new_tokens + t) * a.hq + head;
          const float inv = sum == 0.f ? 0.f : 1.f / sum;
          // this thread's channels: pairs 8 j + 2 c (bf16), or kDT (2 c + y) + j (e4m3)
          if (!kFp8) {
#pragma unroll
            for (int j = 0; j < kDT; ++j) {
              const int ch = 8 * j + 2 * c;
              if (ch >= a.d) continue;
              if (whole) *reinterpret_cast<uint32_t*>(a.out + at * a.d + ch) = pack_bf16(o[mt][j][2 * x] * inv, o[mt][j][2 * x + 1] * inv);
              else *reinterpret_cast<float2*>(p.part_o + (slot * kRows + r) * a.d + ch) = make_float2(o[mt][j][2 * x], o[mt][j][2 * x + 1]);
            }
          } else {
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
              for (int j = 0; j < kDT; j += 4) {
                const int ch = kDT * (2 * c + y) + j;
                if (ch >= a.d) continue;
                const float v[4] = {o[mt][j][2 * x + y], o[mt][j + 1][2 * x + y], o[mt][j + 2][2 * x + y], o[mt][j + 3][2 * x + y]};
                if (whole)
                  *reinterpret_cast<uint2*>(a.out + at * a.d + ch) = make_uint2(pack_bf16(v[0] * inv, v[1] * inv), pack_bf16(v[2] * inv, v[3] * inv));
                else
                  *reinterpret_cast<float4*>(p.part_o + (slot * kRows + r) * a.d + ch) = make_float4(v[0], v[1], v[2], v[3]);
              }
          }
          if (c == 0) {
            if (!whole) p.part_ml[slot * kRows + r] = make_float2(top, sum);
            else if (a.lse)
              a.lse[at] = sum == 0.f ? -INFINITY : ((top == -INFINITY ? 0.f : top) - (kFp8 ? kWeightShift : 0.f) + log2f(sum)) * 0.6931471805599453f;
          }
        }
      if (pieces == 0 && blk > 0 && blk + take == n_blk) {  // this CTA ends a unit that others began
        // the CTA of its first block; the unit is that CTA's first one if its share begins there, or in
        // the end (without blocks) of the unit before
        const int64_t start = w0 - blk;
        const int64_t c0 = ((start + 1) * ctas - 1) / total;
        const int64_t first = 2 * c0 + (start - c0 * total / ctas <= kUnitCost ? 0 : 1);
        meta = make_int4((int)first, (int)(cta - c0 + 1), (int)((int64_t)b * units_per_seq + u), 0);
      }
    }
    ++pieces;
    slot_out = slot_out == 2 ? 0 : slot_out + 1;
  }
  if (warp == kWarps - 1 && lane == 0) p.meta[cta] = meta;
}

// Joins the partial results of every unit that more than one CTA worked on, in the order of its
// keys.  The launch's blocks take (unit, rows) jobs in turn: eight rows, a warp each, where a unit
// has few partials; one row, its partials dealt to the eight warps, where it has many.
constexpr int kJoinThreads = 256;
constexpr int kFewPartials = 8;

__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(const __grid_constant__ DecodeParams p, int ctas, int rows_per_block,
                                                                 float weight_shift) {
  const AttnDecodeArgs& a = p.a;
  __shared__ int s_end[kMaxCtas];      // jobs up to and with CTA i's unit
  __shared__ int4 s_meta[kMaxCtas];
  __shared__ int s_warp[kJoinThreads / 32];
  __shared__ float s_o[kJoinThreads / 32][kAttnMaxDim];
  __shared__ float2 s_ml[kJoinThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  sm100::griddep_wait();
  int jobs[2] = {0, 0};
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = 2 * tid + k;
    if (i < ctas) {
      const int4 mt = p.meta[i];
      s_meta[i] = mt;
      if (mt.y > 0) {
        const int rb = mt.z % p.row_blocks;
        const int live = min(rows_per_block, p.rows - rb * rows_per_block);
        jobs[k] = mt.y > kFewPartials ? live : (live + 7) / 8;
      }
    }
  }
  int incl = jobs[0] + jobs[1];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += t;
  }
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  int before = 0, total = 0;
  for (int w = 0; w < kJoinThreads / 32; ++w) {
    if (w < warp) before += s_warp[w];
    total += s_warp[w];
  }
  const int end1 = before + incl, end0 = end1 - jobs[1];
  if (2 * tid < ctas) s_end[2 * tid] = end0;
  if (2 * tid + 1 < ctas) s_end[2 * tid + 1] = end1;
  __syncthreads();

  for (int job = blockIdx.x; job < total; job += gridDim.x) {
    int lo = 0, hi = ctas - 1;  // the first CTA whose end is beyond the job
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (s_end[mid] > job) hi = mid;
      else lo = mid + 1;
    }
    const int4 mt = s_meta[lo];
    const int local = job - (lo > 0 ? s_end[lo - 1] : 0);
    const int rb = mt.z % p.row_blocks, bh = mt.z / p.row_blocks;
    const int live = min(rows_per_block, p.rows - rb * rows_per_block);
    const bool many = mt.y > kFewPartials;
    const int r = many ? local : local * 8 + warp;
    const int cta0 = mt.x >> 1;
    auto slot = [&](int i) { return (int64_t)(i == 0 ? mt.x : 2 * (cta0 + i)) * rows_per_block + r; };
    float top = -INFINITY, sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < live) {
      const int step = many ? kJoinThreads / 32 : 1;
      for (int i = many ? warp : 0; i < mt.y; i += step) top = fmaxf(top, p.part_ml[slot(i)].x);
#pragma unroll 4
      for (int i = many ? warp : 0; i < mt.y; i += step) {
        const int64_t s = slot(i);
        const float2 ml = p.part_ml[s];
        const float f = ml.x == -INFINITY ? 1.f : ex2_approx(ml.x - top);
        sum = fmaf(ml.y, f, sum);
        if (4 * lane < a.d) {
          const float4 t = *reinterpret_cast<const float4*>(p.part_o + s * a.d + 4 * lane);
          acc.x = fmaf(t.x, f, acc.x); acc.y = fmaf(t.y, f, acc.y);
          acc.z = fmaf(t.z, f, acc.z); acc.w = fmaf(t.w, f, acc.w);
        }
      }
    }
    if (many) {
      __syncthreads();
      reinterpret_cast<float4*>(s_o[warp])[lane] = acc;
      if (lane == 0) s_ml[warp] = make_float2(top, sum);
      __syncthreads();
      if (warp != 0) continue;
      top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kJoinThreads / 32; ++w) top = fmaxf(top, s_ml[w].x);
      sum = 0.f;
      acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kJoinThreads / 32; ++w) {
        const float f = s_ml[w].x == -INFINITY ? 1.f : ex2_approx(s_ml[w].x - top);
        sum = fmaf(s_ml[w].y, f, sum);
        const float4 t = reinterpret_cast<const float4*>(s_o[w])[lane];
        acc.x = fmaf(t.x, f, acc.x); acc.y = fmaf(t.y, f, acc.y);
        acc.z = fmaf(t.z, f, acc.z); acc.w = fmaf(t.w, f, acc.w);
      }
    }
    if (r < live) {
      const int row = rb * rows_per_block + r;
      const int b = bh / a.hkv, h = bh - b * a.hkv;
      const int t = row / p.group, head = h * p.group + row - t * p.group;
      const int64_t at = ((int64_t)b * a.new_tokens + t) * a.hq + head;
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      if (4 * lane < a.d)
        *reinterpret_cast<uint2*>(a.out + at * a.d + 4 * lane) = make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
      if (lane == 0 && a.lse)
        a.lse[at] = sum == 0.f ? -INFINITY : ((top == -INFINITY ? 0.f : top) - weight_shift + log2f(sum)) * 0.6931471805599453f;
    }
  }
}

size_t up256(size_t b) { return (b + 255) / 256 * 256; }

// Rows of one row block: 16 while all rows of a (sequence, kv head) fit, else 32.
int rows_per_block(int rows) { return rows <= 16 ? 16 : 32; }

template <bool kFp8, int kDP, int kMT>
cudaError_t launch_typed(const AttnDecodeArgs& a, cudaStream_t stream) {
  using G = Geo<kFp8, kDP, kMT>;
  using SM = Smem<kFp8, kDP, kMT>;
  static bool attr_done[64] = {};
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  DecodeParams p;
  p.a = a;
  p.group = a.hq / a.hkv;
  p.rows = a.new_tokens * p.group;
  p.row_blocks = (p.rows + SM::kRows - 1) / SM::kRows;
  const int64_t units = (int64_t)a.batch * a.hkv * p.row_blocks;
  const int64_t cap = (int64_t)a.max_pages << a.page_shift;
  const int64_t most_blocks = cap > G::kBlockTok ? (cap + G::kBlockTok - 1) / G::kBlockTok : 1;
  int64_t grid = (int64_t)kCtasPerSm * sms;
  if (grid > kMaxCtas) grid = kMaxCtas;
  if (units < grid && units * most_blocks < grid) grid = units * most_blocks;
  uint8_t* ws = a.workspace;
  p.status = reinterpret_cast<uint32_t*>(ws);
  p.meta = reinterpret_cast<int4*>(ws + kWorkspaceHeader);
  p.part_ml = reinterpret_cast<float2*>(ws + kWorkspaceHeader + up256(kMaxCtas * sizeof(int4)));
  p.part_o = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(p.part_ml) + up256((size_t)2 * kMaxCtas * SM::kRows * sizeof(float2)));
  constexpr uint32_t kSmem = SM::kTotal + 1024;
  cudaError_t e = set_smem_once(attn_decode_kernel<kFp8, kDP, kMT>, kSmem, attr_done);
  if (e != cudaSuccess) return e;
  attn_decode_kernel<kFp8, kDP, kMT><<<(unsigned)grid, kThreads, kSmem, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess || most_blocks == 1) return e;  // (no unit has two blocks: nothing to join)
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * sms));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_join_kernel, p, (int)grid, (int)SM::kRows, kFp8 ? kWeightShift : 0.f);
}

template <bool kFp8, int kDP>
cudaError_t launch_rows(const AttnDecodeArgs& a, cudaStream_t stream) {
  return rows_per_block(a.new_tokens * (a.hq / a.hkv)) == 16 ? launch_typed<kFp8, kDP, 1>(a, stream)
                                                             : launch_typed<kFp8, kDP, 2>(a, stream);
}

}  // namespace

size_t attn_decode_workspace_bytes(int32_t rows, int32_t d) {
  const size_t r = rows_per_block(rows);
  return kWorkspaceHeader + up256(kMaxCtas * sizeof(int4)) + up256(2 * kMaxCtas * r * sizeof(float2)) +
         up256(2 * kMaxCtas * r * (size_t)d * sizeof(float));
}

cudaError_t launch_attn_decode(const AttnDecodeArgs& a, cudaStream_t stream) {
  if ((int64_t)a.batch * a.new_tokens == 0) return cudaSuccess;
  if (a.k_scale) return a.d <= 64 ? launch_rows<true, 64>(a, stream) : launch_rows<true, 128>(a, stream);
  return a.d <= 64 ? launch_rows<false, 64>(a, stream) : launch_rows<false, 128>(a, stream);
}

}  // namespace kda
