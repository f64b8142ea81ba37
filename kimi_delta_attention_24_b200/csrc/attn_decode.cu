// Attention of one or a few new tokens per sequence over the paged key-value cache.
//
// Row r = (new token t, query head) of a sequence and its kv head h sees the keys j of the cache with
// j <= p (p = len - new + t, its own position) and, with a window W, j > p - W:
//     z_j = scale q . K_j,  capped: z = cap tanh(z / cap);   o = sum_j e^{z_j} V_j / sum_j e^{z_j}
// with the running maximum m and sum l of the softmax (base 2).
//
// What bounds it: a key and value row is read once for every 16 of the G T rows that use it (G query heads per
// kv head, T new tokens), 4 flops per row and 2 x 2 bytes (bf16).  Up to 8 rows that is HBM; from 9 on, with a cap
// or an e4m3 cache first, the latency of dependent instructions.  So the design is a stream of cache tiles
// with little else:
//   - Split: the (sequence, kv head, row block) units are laid end to end as blocks of one tile of keys
//     per warp, and every CTA (two or three per SM) takes an equal share of all blocks, wherever it
//     begins and ends, so ragged lengths cost no balance.  A unit that several CTAs share leaves fp32
//     partial results (o, m, l) in the workspace, joined in a fixed order by a second, dependent launch.
//   - Each of a CTA's warps streams its own tiles (one per block) through its own ring of stages, with
//     no CTA barrier: 16-byte cp.async copies into swizzled rows (conflict-free matrix loads), under way
//     also across the ends of units; about 130 KB of copies in flight per SM.  (TMA boxes instead cost
//     the issuing warp 800 to 900 cycles a tile, four boxes each, of 2600 to 3500.)
//   - The warps' results of a unit meet as a chain through shared memory, so that no warp waits for a
//     slower one before it goes on with the next unit.  With very many units each warp takes a share of
//     its own instead; few short units are not split at all.
//   - The products are transposed, S^T = K Q^T and O^T = V^T P^T, mma.sync m16n8k16 with the keys (the
//     channels) as the 16 and 8 rows of queries as the 8: a unit of up to 8 rows (one kv head's group
//     at T = 1) wastes half as much of each instruction, and half the registers, as with 16 rows.
//   - What remains to be hidden is latency: two or three warps per scheduler take 2600 to 3500 cycles a tile
//     whether its bytes have arrived or not.  So dependent products are kept apart, and the softmax
//     exchanges maxima between threads only when a score passes its row's reference by 2^8 (e4m3 cache: 2).
//   - bf16 cache: P enters the second product as a bf16 pair hi + lo, so its rounding (2^-17) stays
//     below that of the bf16 output.  e4m3 cache: codes are exact in fp16; the key's scale multiplies
//     the score, and the value's enters the exponent, w_j = 2^(z_j + log2 s_j - M) with M the row's
//     reference of that sum (within 2 of its maximum); times 2^14 it is rounded to fp16 (2^-11 down to
//     2^-28 of 2^M, at worst by 2^-39 of it; moving M only past 2^8, times 2^7, costs 2^7 of that and saves 1.5 us
//     of 175.4 at 8 sequences to 131072, 0.4 of 32.8 at 48 to 8192).  The row's sum adds w_j / s_j in fp32 before that
//     rounding.  q (bf16) is scaled by a power of two per row to fit fp16.
#include <cuda_fp16.h>

#include <algorithm>

#include "attn_common.cuh"
#include "kda_device.cuh"

namespace kda {
namespace {

// How the work is dealt out: equal shares of all blocks to the CTAs (kCommon), or to their warps, where
// units are very many (kSolo); or each unit to one CTA, where they are few and short (kWhole).
enum Mode { kCommon, kSolo, kWhole };

constexpr int kMaxSms = 160;               // bound used for the workspace (148 on a B200)
constexpr int kMaxShares = kMaxSms * 2 * 4;  // (kSolo)
// How far (base 2) a score passes a row's reference before it moves, by the type of cache: fp32 weights
// may grow; fp16 weights, times 2^kWeightShift, go up to 2^15, and what they may grow is lost at their lower end.
constexpr float kLazyBf16 = 8.0f, kLazyE4m3 = 1.0f;
constexpr float kWeightShift = 14.0f;
constexpr float kScaleLeast = 0x1p-80f;  // of a value row

struct DecodeParams {
  AttnDecodeArgs a;
  int32_t group, rows, row_blocks;  // rows = new_tokens * group, of one (sequence, kv head)
  float4* part_o;                   // [2 * shares][row tile][channel tile][lane]: as the product leaves it
  float4* part_ml;                  // [2 * shares][row tile][lane]: (m, l) of the lane's two rows
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
// An 8 x 8 matrix of 16-bit elements transposed among the lanes (lane: row lane / 4, columns 2 (lane % 4) + {0, 1}).
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
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
__device__ __forceinline__ float tanh_near(float x) {
  const float q = x * x;
  return x * fmaf(q, q + 105.f, 945.f) * rcp_approx(fmaf(q, fmaf(q, 15.f, 420.f), 945.f));
}
__device__ __forceinline__ float tanh_any(float x) {
  const float far = fmaf(-2.f, rcp_approx(ex2_approx(x * (2.f * kLog2e)) + 1.f), 1.f);
  return fabsf(x) < 1.f ? tanh_near(x) : far;
}

// Tile geometry.  kDP: the head size padded to 64 or 128 channels (the padding is zero in q and in
// the loaded rows); kNQ: tiles of 8 rows per unit (1 or 2); kTok: keys of one warp's tile, 8 KB of K and V
// together (4 KB for 64 e4m3 channels); a block is one tile per warp.  Two CTAs of 4 warps per SM:
// at 128 channels their registers allow no more beyond 8 rows; up to 8, more warps (two CTAs of 6, three of
// 4) were no faster for long sequences and slower for short ones.  The bf16 cache has room for a third stage
// there, and needs the stages more than a third CTA at 64 channels (4 rows: 51.1 us with two, 51.6 with three).
template <bool kFp8, int kDP, int kNQ, Mode kMode>
struct Geo {
  static constexpr int kWarps = kMode == kWhole ? 8 : 4;
  static constexpr int kThreads = 32 * kWarps;
  // CTAs per SM: three at 64 e4m3 channels, whose tiles are small (64 sequences to 4096: 4 rows of 8 kv heads
  // 43.0 us with two and 38.9 with three, 12 rows of 4 heads 35.1 and 33.2)
  static constexpr int kCtas = kMode == kWhole ? 1 : kMode == kCommon && kDP == 64 && kFp8 ? 3 : 2;
  static constexpr int kMaxCtas = kMaxSms * kCtas;
  static constexpr int kTok = kFp8 ? 32 : (kDP == 128 ? 16 : 32);
  static constexpr int kRowBytes = kFp8 ? kDP : 128;               // bytes of a row in one column block
  static constexpr int kColBlocks = kFp8 ? 1 : kDP / 64;           // 128-byte column blocks (bf16)
  static constexpr int kOpBytes = kTok * kRowBytes * kColBlocks;   // K (or V) of one tile
  static constexpr int kStageBytes = 2 * kOpBytes;
  static constexpr int kWarpBytes = kCtas == 3 ? 12288 : kNQ == 1 && !kFp8 ? 24576 : 16384;
  static constexpr int kStages = kWarpBytes / kStageBytes;
  static constexpr int kShares = kMode == kSolo ? kWarps : 1;      // shares of a CTA
  static constexpr int kBlockTok = kTok * (kMode == kSolo ? 1 : kWarps);
  static constexpr int kScaleBytes = kFp8 ? 3 * kTok * 4 : 0;      // k scales; v scales, then their logarithms; reciprocals
};

// Byte offset of 16-byte chunk `chunk` of row `row` in a swizzled block of kRowBytes-wide rows.
template <int kRowBytes>
__device__ __forceinline__ uint32_t swz(uint32_t row, uint32_t chunk) {
  return kRowBytes == 128 ? row * 128 + ((chunk ^ (row & 7)) << 4) : row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4);
}

// a / b for 0 <= a, 0 < b: by 32 bits where they suffice.
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// Keys [lo, hi) that any row of a sequence sees.
__device__ __forceinline__ void key_range(const AttnDecodeArgs& a, int len, int& lo, int& hi, uint32_t* status) {
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
// the next unit, until the share is used up.  lens: the lengths in shared memory, or null where there are
// more than kLens (a load from global memory waits behind all the copies under way).
constexpr int kLens = 512;
template <int kBlockTok>
struct Walk {
  int64_t left;                          // cost left in the share
  int b, u, lo, len, n_blk, blk, take;   // the piece
  int pos;                               // the cursor behind it, in the unit's cost (its blocks come first)
  __device__ __forceinline__ void to_sequence(const AttnDecodeArgs& a, const int* lens) {
    key_range(a, lens ? lens[b] : a.seq_lens[b], lo, len, nullptr);
    n_blk = num_blocks<kBlockTok>(lo, len);
  }
  // To position `off` of sequence `first`.
  __device__ __forceinline__ void begin(const AttnDecodeArgs& a, const int* lens, int first, int64_t off) {
    b = first;
    to_sequence(a, lens);
    u = (int)divide(off, n_blk + kUnitCost);
    pos = (int)(off - (int64_t)u * (n_blk + kUnitCost));
  }
  __device__ __forceinline__ bool next(const AttnDecodeArgs& a, const int* lens, int64_t units_per_seq) {
    while (left > 0) {
      if (pos == n_blk + kUnitCost) {
        pos = 0;
        if (++u == units_per_seq) {
          u = 0;
          ++b;
          to_sequence(a, lens);
        }
      }
      blk = pos;
      const int step = (int)min((int64_t)(n_blk + kUnitCost - blk), left);
      take = min(n_blk - blk, step);
      left -= step;
      pos += step;
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

template <bool kFp8, int kDP, int kNQ, Mode kMode>
struct Smem {
  using G = Geo<kFp8, kDP, kNQ, kMode>;
  static constexpr int kWarps = G::kWarps;
  static constexpr int kQPlaces = kMode == kSolo ? 2 * kWarps : 3;  // two of each warp, or three of all
  static constexpr int kRows = 8 * kNQ, kDM = kDP / 16;
  static constexpr int kQRowBytes = kRows * kDP * 2;                // one unit's queries as they are
  static constexpr int kScaleOff = kWarps * G::kWarpBytes;          // (the rings come first)
  static constexpr int kQOff = kScaleOff + kWarps * G::kStages * G::kScaleBytes;
  static constexpr int kSumOff = kQOff + kQPlaces * kQRowBytes;         // the warps' sum,
  static constexpr int kMlOff = kSumOff + (kMode == kSolo ? 0 : kNQ * kDM * 32 * 16);  // and each row's maximum and sum
  static constexpr int kScanOff = kMlOff + (kMode == kSolo ? 0 : kNQ * 32 * 16);       // one int64 per warp
  static constexpr int kTotal = kScanOff + 8 * kWarps;
};

// Rows of one row tile (o / l) to the output: o[jj] as the product leaves it, channel tile jj, the
// lane's rows 2 c + {0, 1}; inv their 1 / l.  row_out: the output row of tile row lane / 4, or null.
template <bool kFp8, int kDP>
__device__ __forceinline__ void write_tile(const float (&o)[4], int jj, const float (&inv)[2], __nv_bfloat16* row_out, int d) {
  const int c = threadIdx.x & 3;
  // after the transposition a lane holds two channels of row lane / 4
  const uint32_t t0 = transpose8(pack_bf16(o[0] * inv[0], o[1] * inv[1]));
  const uint32_t t1 = transpose8(pack_bf16(o[2] * inv[0], o[3] * inv[1]));
  // bf16: channels 16 jj + 2 c + {0, 1}, and 8 further; e4m3: (kDP / 8) (2 c) + 2 jj and (kDP / 8) (2 c + 1) + 2 jj, each with the next
  const int ch0 = kFp8 ? (kDP / 8) * 2 * c + 2 * jj : 16 * jj + 2 * c, ch1 = ch0 + (kFp8 ? kDP / 8 : 8);
  if (row_out && ch0 < d) *reinterpret_cast<uint32_t*>(row_out + ch0) = kFp8 ? __byte_perm(t0, t1, 0x5410) : t0;
  if (row_out && ch1 < d) *reinterpret_cast<uint32_t*>(row_out + ch1) = kFp8 ? __byte_perm(t0, t1, 0x7632) : t1;
}
__device__ __forceinline__ float lse_of(float m, float l, float shift) {
  return l == 0.f ? -INFINITY : ((m == -INFINITY ? 0.f : m) - shift + log2f(l)) * 0.6931471805599453f;
}

template <bool kFp8, int kDP, int kNQ, Mode kMode>
__global__ void __launch_bounds__(Geo<kFp8, kDP, kNQ, kMode>::kThreads, Geo<kFp8, kDP, kNQ, kMode>::kCtas)
    attn_decode_kernel(const __grid_constant__ DecodeParams p) {
  using G = Geo<kFp8, kDP, kNQ, kMode>;
  using SM = Smem<kFp8, kDP, kNQ, kMode>;
  constexpr int kWarps = G::kWarps, kThreads = G::kThreads;
  constexpr int kTok = G::kTok, kKT = kTok / 16, kKS = kDP / 16, kDM = SM::kDM, kRows = SM::kRows;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((128 - (sm100::smem_u32(smem_raw) & 127)) & 127);
  const AttnDecodeArgs& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  uint8_t* stages = smem + warp * G::kWarpBytes;
  float* scales = reinterpret_cast<float*>(smem + SM::kScaleOff) + warp * G::kStages * (G::kScaleBytes / 4);
  float4* s_sum = reinterpret_cast<float4*>(smem + SM::kSumOff) + lane;
  float4* s_ml = reinterpret_cast<float4*>(smem + SM::kMlOff) + lane;
  __shared__ int s_any;
  int64_t* s_scan = reinterpret_cast<int64_t*>(smem + SM::kScanOff);
  __shared__ int s_b[G::kShares];
  __shared__ int64_t s_off[G::kShares];
  __shared__ int s_len[kMode == kWhole ? 1 : kLens];
  const int* lens = kMode != kWhole && a.batch <= kLens ? s_len : nullptr;

  // (this launch may begin while the one before it drains, and the join while this one does: each
  // waits here for all that ran before)
  sm100::griddep_wait();
  sm100::griddep_launch_dependents();

  const int64_t units_per_seq = (int64_t)a.hkv * p.row_blocks;
  Walk<G::kBlockTok> in, out;  // the pieces whose tiles this warp loads next, and computes next
  int64_t share = blockIdx.x;
  if (kMode == kWhole) {
    // (the lengths of all sequences are only looked at for the status)
    if (blockIdx.x == 0)
      for (int b = tid; b < a.batch; b += kThreads) {
        int lo, hi;
        key_range(a, a.seq_lens[b], lo, hi, p.status);
      }
    in.begin(a, nullptr, (int)(share / units_per_seq), 0);
    in.u = (int)(share - in.b * units_per_seq);
    in.left = in.n_blk;
    if (tid == 0) s_any = 0;
    __syncthreads();
  } else {
    // ---- this CTA's share [w0, w1) of all blocks, and the sequence it begins in
    const int per = (a.batch + kThreads - 1) / kThreads;
    const int b_first = tid * per, b_last = min(a.batch, b_first + per);
    int64_t mine = 0;
    for (int b = b_first; b < b_last; ++b) {
      int lo, hi;
      const int len = a.seq_lens[b];
      if (b < kLens) s_len[b] = len;
      key_range(a, len, lo, hi, blockIdx.x == 0 ? p.status : nullptr);
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
    const int64_t shares = min(total, (int64_t)gridDim.x * G::kShares);
    if ((int64_t)blockIdx.x * G::kShares >= shares) return;
#pragma unroll 1
    for (int k = 0; k < G::kShares; ++k) {
      const int64_t first = divide(((int64_t)blockIdx.x * G::kShares + k) * total, shares);
      if (mine > 0 && before <= first && first < before + mine) {
        int64_t at = before;
        for (int b = b_first; b < b_last; ++b) {
          int lo, hi;
          key_range(a, lens ? lens[b] : a.seq_lens[b], lo, hi, nullptr);
          const int64_t n = (num_blocks<G::kBlockTok>(lo, hi) + kUnitCost) * units_per_seq;
          if (first < at + n) {
            s_b[k] = b;
            s_off[k] = first - at;
            break;
          }
          at += n;
        }
      }
    }
    __syncthreads();
    share = (int64_t)blockIdx.x * G::kShares + (kMode == kSolo ? warp : 0);
    if (share >= shares) return;
    in.left = divide((share + 1) * total, shares) - divide(share * total, shares);
    in.begin(a, lens, s_b[kMode == kSolo ? warp : 0], s_off[kMode == kSolo ? warp : 0]);
  }
  out = in;

  const int page_mask = (1 << a.page_shift) - 1;
  // scores to base 2 (to the cap's units): a positive factor, its sign goes to the queries, so that
  // maxima can be taken before it (a scale of zero: zero queries; else a normal number, by the host's check)
  const float base_scale = a.scale == 0.f ? 1.f : fabsf(a.softcap > 0.f ? a.scale / a.softcap : a.scale * kLog2e);
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
  constexpr int kPlaces = kMode == kSolo ? 2 : 3;  // for queries, used in turn
  uint8_t* q_places = smem + SM::kQOff + (kMode == kSolo ? warp * 2 * SM::kQRowBytes : 0);
  int in_piece = -1, in_slot = kPlaces - 1, ahead = 0;  // the piece being loaded, its place for queries; tiles under way
  bool in_more = true, in_first = false;
  // To the next tile, and the page numbers ahead of it.  Where a tile lies in one page, lane t holds
  // that of tile in_batch + t, 32 tiles from one load (a load per tile, waited for behind the copies
  // under way, took 350 to 750 cycles of it); else the lane holds that of the key it stands for.  Either
  // is the page of the nearest key in [lo, len).
  int in_batch = 0;
  auto advance = [&]() {
    ++in_i;
    bool fresh = !one_page || in_i - in_batch == 32;
    while (in_i >= in_end) {
      in_more = in.next(a, lens, units_per_seq);
      if (!in_more) return;
      ++in_piece;
      in_slot = in_slot == kPlaces - 1 ? 0 : in_slot + 1;
      in_first = true;
      in_h = in.u / p.row_blocks;
      in.tiles(kMode == kSolo ? 0 : warp, kTok, in_tok, in_i, in_end);
      fresh = true;
    }
    if (!fresh) return;
    in_batch = in_i;
    int64_t tok = in_tok + (int64_t)(one_page ? min(in_i + lane, in_end - 1) : in_i) * G::kBlockTok + (one_page ? 0 : lane & (kTok - 1));
    tok = tok < in.lo ? in.lo : (tok >= in.len ? in.len - 1 : tok);
    page_next = a.page_table[(int64_t)in.b * a.max_pages + (tok >> a.page_shift)];
  };
  // the copies of the next tile, as one group
  auto issue = [&]() {
    {
      int page = one_page ? __shfl_sync(0xffffffffu, page_next, in_i - in_batch) : page_next;
      if ((uint32_t)page >= (uint32_t)a.num_pages) {  // never read outside the cache
        if (p.status) atomicOr(p.status, kStatusBadIndex);
        page = 0;
      }
      const int t0 = in_tok + in_i * G::kBlockTok;
      const uint32_t st = ring + stage_in * G::kStageBytes;
      if (in_first) {
        // the unit's queries come with its first tile: a load that is waited for at the unit's start
        // would queue behind all the copies under way.  All warps of a shared unit copy them (the
        // same bytes); of three places the one behind a warp that lags and before one that leads is free.
        in_first = false;
        constexpr int kQChunks = kDP * 2 / 16, kQPass = 32 / kQChunks;
        const int base = (in.u - in_h * p.row_blocks) * kRows, ch = lane % kQChunks;
        const int live = min(kRows, p.rows - base);
        const uint32_t dst = sm100::smem_u32(q_places + in_slot * SM::kQRowBytes);
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
        constexpr int kFullPass = kPass * kDP * (kFp8 ? 1 : 2);
        if (kPass * row_bytes == kFullPass) {  // (the steps as constants)
#pragma unroll
          for (int i = 0; i < kTok / kPass; ++i) copy_rows(i, ks + i * kFullPass, vs + i * kFullPass);
        } else {
#pragma unroll
          for (int i = 0; i < kTok / kPass; ++i) {
            copy_rows(i, ks, vs);
            ks += kPass * row_bytes;
            vs += kPass * row_bytes;
          }
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

  int pieces = 0, slot_out = 0;
  bool more = out.next(a, lens, units_per_seq);
  while (more) {
    const int b = out.b, len = out.len, lo = out.lo, blk = out.blk, take = out.take, n_blk = out.n_blk, u = out.u;
    const int h = u / p.row_blocks, row_base = (u - h * p.row_blocks) * kRows;
    int tok0, i_begin, i_end;
    out.tiles(kMode == kSolo ? 0 : warp, kTok, tok0, i_begin, i_end);
    more = out.next(a, lens, units_per_seq);

    // ---- the rows' key ranges, their queries as fragments.  A lane works on the scores of rows
    // 2 c + {0, 1} of each row tile, and holds the queries of row g.
    uint32_t qf[kNQ][kKS][2];
    float rscale[kNQ][2];   // score factor of the lane's rows
    int row_hi[kNQ][2], row_lo[kNQ][2];
#pragma unroll
    for (int nq = 0; nq < kNQ; ++nq)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int r = row_base + nq * 8 + 2 * c + x;
        const int pos = len - a.new_tokens + r / p.group;
        row_hi[nq][x] = r < p.rows ? pos + 1 : 0;
        row_lo[nq][x] = a.window > 0 && pos >= a.window ? pos - a.window + 1 : 0;
        rscale[nq][x] = base_scale;
      }
    auto make_fragments = [&]() {
      const uint8_t* q_rows = q_places + slot_out * SM::kQRowBytes;
#pragma unroll
      for (int nq = 0; nq < kNQ; ++nq) {
        const uint8_t* q_row = q_rows + (8 * nq + g) * (kDP * 2);
        auto load16 = [&](int ch) { return *reinterpret_cast<const uint4*>(q_row + (((ch / 8) ^ g) << 4)); };
        auto load4 = [&](int ch) { return *reinterpret_cast<const uint32_t*>(q_row + (((ch / 8) ^ g) << 4) + (ch % 8) * 2); };
        // (rows beyond the unit's are zero: their scores would else move references and pass the cap)
        const uint32_t keep = row_base + nq * 8 + g < p.rows ? q_keep : 0u, sign = keep & q_sign;
        uint32_t (&f)[kKS][2] = qf[nq];
        if (!kFp8) {
#pragma unroll
          for (int ks = 0; ks < kKS; ++ks) {
            f[ks][0] = (load4(16 * ks + 2 * c) & keep) ^ sign;
            f[ks][1] = (load4(16 * ks + 8 + 2 * c) & keep) ^ sign;
          }
        } else {
          // channels 64 j + 16 c + 4 s + {0..3} are k-step 4 j + s of this lane (as the key bytes are read)
          uint32_t wv[kDP / 64][8];
          float big = 0.f;
#pragma unroll
          for (int j = 0; j < kDP / 64; ++j) {
            const uint4 v0 = load16(64 * j + 16 * c), v1 = load16(64 * j + 16 * c + 8);
            wv[j][0] = v0.x; wv[j][1] = v0.y; wv[j][2] = v0.z; wv[j][3] = v0.w;
            wv[j][4] = v1.x; wv[j][5] = v1.y; wv[j][6] = v1.z; wv[j][7] = v1.w;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              wv[j][i] = (wv[j][i] & keep) ^ sign;
              const float2 t = unpack_bf16(wv[j][i]);
              big = fmaxf(big, fmaxf(fabsf(t.x), fabsf(t.y)));
            }
          }
          big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
          big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
          // the power of two below the row's largest magnitude, whose inverse is a normal number too (exact
          // factors; a row with an infinity or NaN is that whatever the factor)
          int e = (int)((__float_as_uint(big) >> 23) & 255) - 127;
          e = big == 0.f || e > 127 ? 0 : min(max(e, -100), 126);
          const float down = __uint_as_float((uint32_t)(127 - e) << 23), up = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
          for (int x = 0; x < 2; ++x) rscale[nq][x] = base_scale * __shfl_sync(0xffffffffu, up, 4 * (2 * c + x));
#pragma unroll
          for (int j = 0; j < kDP / 64; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float2 t = unpack_bf16(wv[j][i]);
              f[4 * j + i / 2][i & 1] = pack_half(t.x * down, t.y * down);
            }
        }
      }
    };

    float o[kNQ][kDM][4];         // O^T: rows 2 c + (e & 1); channels 16 jj + g + 8 (e >> 1), or (kDP / 8) g + 2 jj + (e >> 1) (e4m3)
    float m[kNQ][2], l[kNQ][2];
#pragma unroll
    for (int nq = 0; nq < kNQ; ++nq) {
#pragma unroll
      for (int j = 0; j < kDM; ++j) o[nq][j][0] = o[nq][j][1] = o[nq][j][2] = o[nq][j][3] = 0.f;
      m[nq][0] = m[nq][1] = -INFINITY;
      l[nq][0] = l[nq][1] = 0.f;
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
      if (i == i_begin) make_fragments();
      uint8_t* st = stages + stage_out * G::kStageBytes;
      const uint32_t ks_addr = sm100::smem_u32(st), vs_addr = ks_addr + G::kOpBytes;
      float* sc = scales + stage_out * 3 * kTok;
      if (kFp8) {
        // once per key: the logarithm of its value scale and the reciprocal.  (A scale that is not a
        // number makes the rows that see its key so, by way of the logarithm; its reciprocal stays
        // finite, for the rows that do not see it.  Scales below 2^-80, which no write to the cache makes, count
        // as that: 2^15 w_j / s_j of 2^30 keys add up to less than fp32's largest.)
        const float v = sc[kTok + lane];
        sc[kTok + lane] = lg2_approx(v < kScaleLeast ? kScaleLeast : v);
        sc[2 * kTok + lane] = rcp_approx(fmaxf(v, kScaleLeast));
        __syncwarp();
      }
      const int t0 = tok0 + i * G::kBlockTok;
      const bool edge = t0 + kTok > all_hi || t0 < all_lo;

      // ---- S^T = K Q^T: element e of s[kt][nq] is key 16 kt + g + 8 (e >> 1), row 2 c + (e & 1).
      // Few sums are kept in several parts, so that a product does not wait for the one before.
      constexpr int kParts = kKT * kNQ == 1 ? 4 : kKT * kNQ == 2 ? 2 : 1;
      float sp[kParts][kKT][kNQ][4] = {};
      if (!kFp8) {
        const uint32_t mrow = (((lane >> 3) & 1) << 3) + (lane & 7), mchunk = lane >> 4;
#pragma unroll
        for (int ks = 0; ks < kKS; ++ks)
#pragma unroll
          for (int kt = 0; kt < kKT; ++kt) {
            uint32_t ka[4];
            ldsm4(ka, ks_addr + (ks >> 2) * (kTok * 128) + swz<128>(kt * 16 + mrow, (ks & 3) * 2 + mchunk));
#pragma unroll
            for (int nq = 0; nq < kNQ; ++nq) {
              mma16816<false>(sp[ks % kParts][kt][nq], ka, qf[nq][ks][0], qf[nq][ks][1]);
            }
          }
      } else {
#pragma unroll
        for (int j = 0; j < kDP / 64; ++j) {
          uint4 kb[kKT][2];
#pragma unroll
          for (int kt = 0; kt < kKT; ++kt)
#pragma unroll
            for (int x = 0; x < 2; ++x) kb[kt][x] = *reinterpret_cast<const uint4*>(st + swz<G::kRowBytes>(kt * 16 + 8 * x + g, 4 * j + c));
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4)
#pragma unroll
            for (int kt = 0; kt < kKT; ++kt) {
              auto word = [&](int x) { return q4 == 0 ? kb[kt][x].x : q4 == 1 ? kb[kt][x].y : q4 == 2 ? kb[kt][x].z : kb[kt][x].w; };
              uint32_t ka[4];
              e4m3x4_to_half2(word(0), ka[0], ka[2]);
              e4m3x4_to_half2(word(1), ka[1], ka[3]);
#pragma unroll
              for (int nq = 0; nq < kNQ; ++nq) {
                mma16816<true>(sp[q4 % kParts][kt][nq], ka, qf[nq][4 * j + q4][0], qf[nq][4 * j + q4][1]);
              }
            }
        }
      }
      float (&s)[kKT][kNQ][4] = sp[0];
#pragma unroll
      for (int part = 1; part < kParts; ++part)
#pragma unroll
        for (int kt = 0; kt < kKT; ++kt)
#pragma unroll
          for (int nq = 0; nq < kNQ; ++nq)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[kt][nq][e] += sp[part][kt][nq][e];

      // ---- scores, masks, the value scales' logarithms.  S becomes z (times the row's factor where it
      // is not yet applied: bf16 without a cap).
      float kf[kKT][2], lv[kKT][2], inv_vs[kFp8 ? kKT : 1][2];
#pragma unroll
      for (int kt = 0; kt < kKT; ++kt)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int key = kt * 16 + g + 8 * y;
          kf[kt][y] = kFp8 ? sc[key] : 1.f;
          lv[kt][y] = kFp8 ? sc[kTok + key] : 0.f;
          if (kFp8) inv_vs[kFp8 ? kt : 0][y] = sc[2 * kTok + key];
        }
      const bool capped = a.softcap > 0.f;
      if (capped) {
        // in the cap's units; scores beyond it are rare: the shorter form of the tangent for all, unless
        // there is one
        const float cap2 = a.softcap * kLog2e;
        float most = 0.f;
#pragma unroll
        for (int kt = 0; kt < kKT; ++kt)
#pragma unroll
          for (int nq = 0; nq < kNQ; ++nq)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float& z = s[kt][nq][e];
              z *= kFp8 ? kf[kt][e >> 1] * rscale[nq][e & 1] : rscale[nq][e & 1];
              most = fmaxf(most, fabsf(z));
            }
        if (__any_sync(0xffffffffu, most >= 1.f)) {
#pragma unroll
          for (int kt = 0; kt < kKT; ++kt)
#pragma unroll
            for (int nq = 0; nq < kNQ; ++nq)
#pragma unroll
              for (int e = 0; e < 4; ++e) s[kt][nq][e] = fmaf(cap2, tanh_any(s[kt][nq][e]), lv[kt][e >> 1]);
        } else {
#pragma unroll
          for (int kt = 0; kt < kKT; ++kt)
#pragma unroll
            for (int nq = 0; nq < kNQ; ++nq)
#pragma unroll
              for (int e = 0; e < 4; ++e) s[kt][nq][e] = fmaf(cap2, tanh_near(s[kt][nq][e]), lv[kt][e >> 1]);
        }
      } else if (kFp8) {
#pragma unroll
        for (int kt = 0; kt < kKT; ++kt)
#pragma unroll
          for (int nq = 0; nq < kNQ; ++nq)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[kt][nq][e] = fmaf(s[kt][nq][e] * kf[kt][e >> 1], rscale[nq][e & 1], lv[kt][e >> 1]);
      }
      if (edge) {
#pragma unroll
        for (int kt = 0; kt < kKT; ++kt)
#pragma unroll
          for (int nq = 0; nq < kNQ; ++nq)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int j = t0 + kt * 16 + g + 8 * (e >> 1);
              if (j >= row_hi[nq][e & 1] || j < row_lo[nq][e & 1]) s[kt][nq][e] = -INFINITY;
            }
      }
      // ---- running sum and reference of the exponents; P in place of S.  The reference m of a row is
      // its maximum when it was last moved: it moves (for all rows of the warp) only when a score
      // passes it by kLazy, so P stays below 2^kLazy (e4m3: 2^15 with its shift) and most tiles need no exchange between lanes.
      float mx[kNQ][2];
      bool passed = false;
#pragma unroll
      for (int nq = 0; nq < kNQ; ++nq)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          mx[nq][x] = -INFINITY;
#pragma unroll
          for (int kt = 0; kt < kKT; ++kt) mx[nq][x] = fmaxf(mx[nq][x], fmaxf(s[kt][nq][x], s[kt][nq][x + 2]));
          mx[nq][x] *= kFp8 || capped ? 1.f : rscale[nq][x];
          passed |= mx[nq][x] > m[nq][x] + (kFp8 ? kLazyE4m3 : kLazyBf16);
        }
      if (__any_sync(0xffffffffu, passed)) {
#pragma unroll
        for (int nq = 0; nq < kNQ; ++nq) {
          float alpha[2];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float t = mx[nq][x];
#pragma unroll
            for (int sh = 4; sh < 32; sh <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, sh));
            const float mn = fmaxf(m[nq][x], t);
            alpha[x] = ex2_approx(m[nq][x] - (mn == -INFINITY ? 0.f : mn));
            m[nq][x] = mn;
            l[nq][x] *= alpha[x];
          }
#pragma unroll
          for (int j = 0; j < kDM; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[nq][j][e] *= alpha[e & 1];
        }
      }
#pragma unroll
      for (int nq = 0; nq < kNQ; ++nq)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float fac = kFp8 || capped ? 1.f : rscale[nq][x];
          const float shift = (m[nq][x] == -INFINITY ? 0.f : m[nq][x]) - (kFp8 ? kWeightShift : 0.f);
#pragma unroll
          for (int kt = 0; kt < kKT; ++kt)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const float z = s[kt][nq][x + 2 * y];
              const float pr = ex2_approx(kFp8 ? z - shift : fmaf(z, fac, -shift));
              s[kt][nq][x + 2 * y] = pr;
              l[nq][x] = kFp8 ? fmaf(pr, inv_vs[kFp8 ? kt : 0][y], l[nq][x]) : l[nq][x] + pr;
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
            if (lane < kRowChunks) {
              const uint4 v = *at;
              const uint32_t wv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int x = 0; x < 4; ++x) odd |= (wv[x] & 0x7f80u) == 0x7f80u || (wv[x] & 0x7f800000u) == 0x7f800000u;
            }
            if (!__any_sync(0xffffffffu, odd)) continue;
#pragma unroll
            for (int nq = 0; nq < kNQ; ++nq)
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                uint32_t bits = 0;  // P of key r and this lane's row, held by lane 4 (r % 8) + c (masks: no local array)
#pragma unroll
                for (int kt = 0; kt < kKT; ++kt) {
                  const uint32_t here = kt == r / 16 ? 0xffffffffu : 0u, second = (r & 8) ? 0xffffffffu : 0u;
                  bits |= here & ((second & __float_as_uint(s[kt][nq][x + 2])) | (~second & __float_as_uint(s[kt][nq][x])));
                }
                const float pr = __uint_as_float(__shfl_sync(0xffffffffu, bits, 4 * (r & 7) + c));
                if (j < row_hi[nq][x] && j >= row_lo[nq][x]) {
#pragma unroll
                  for (int jj = 0; jj < kDM; ++jj)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {  // channel 16 jj + 8 y + g
                      const int chunk = 2 * jj + y;
                      const uint16_t v = *reinterpret_cast<const uint16_t*>(st + G::kOpBytes + (chunk / 8) * (kTok * 128) + swz<128>(r, chunk % 8) + 2 * g);
                      o[nq][jj][x + 2 * y] = fmaf(pr, __uint_as_float((uint32_t)v << 16), o[nq][jj][x + 2 * y]);
                    }
                }
              }
            __syncwarp();
            if (lane < kRowChunks) *at = make_uint4(0, 0, 0, 0);
          }
        }
        __syncwarp();
      }

      // ---- O^T += V^T P^T
#pragma unroll
      for (int kt = 0; kt < kKT; ++kt) {
        uint32_t ph[kNQ][2], pl[kNQ][2];
#pragma unroll
        for (int nq = 0; nq < kNQ; ++nq)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            if (kFp8) {
              ph[nq][y] = transpose8(pack_half(s[kt][nq][2 * y], s[kt][nq][2 * y + 1]));
            } else {
              uint32_t hi, lo2;
              split2(s[kt][nq][2 * y], s[kt][nq][2 * y + 1], hi, lo2);
              ph[nq][y] = transpose8(hi);
              pl[nq][y] = transpose8(lo2);
            }
          }
        if (!kFp8) {
          // (four loads, then their products, hi before lo: a sum is met again after the others)
          const uint32_t vrow = ((lane >> 4) << 3) + (lane & 7), vchunk = (lane >> 3) & 1;
#pragma unroll
          for (int j4 = 0; j4 < kDM / 4; ++j4) {
            uint32_t va[4][4];
#pragma unroll
            for (int q = 0; q < 4; ++q) ldsm4t(va[q], vs_addr + j4 * (kTok * 128) + swz<128>(kt * 16 + vrow, 2 * q + vchunk));
#pragma unroll
            for (int part = 0; part < 2; ++part)
#pragma unroll
              for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int nq = 0; nq < kNQ; ++nq)
                  mma16816<false>(o[nq][4 * j4 + q], va[q], part ? pl[nq][0] : ph[nq][0], part ? pl[nq][1] : ph[nq][1]);
          }
        } else {
          // row g (g + 8) of product tile jj stands for channel (kDP / 8) g + 2 jj (and the next): a lane's
          // bytes of a key are contiguous
          const uint8_t* vst = st + G::kOpBytes;
          constexpr int kWords = kDP / 32;  // 32-bit words of a key per lane: 4 or 2
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
              uint32_t va[4];
              e4m3x4_to_half2(__byte_perm(vw[0][x], vw[1][x], y ? 0x7362 : 0x5140), va[0], va[1]);
              e4m3x4_to_half2(__byte_perm(vw[2][x], vw[3][x], y ? 0x7362 : 0x5140), va[2], va[3]);
#pragma unroll
              for (int nq = 0; nq < kNQ; ++nq) mma16816<true>(o[nq][2 * x + y], va, ph[nq][0], ph[nq][1]);
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
    // (a row's eight lanes hold parts of its sum l)
#pragma unroll
    for (int nq = 0; nq < kNQ; ++nq)
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) l[nq][x] += __shfl_xor_sync(0xffffffffu, l[nq][x], sh);
    // (A warp with a share of its own has the result already.  With one unit per CTA nothing is to go on
    // with: the warps lay their sums side by side over the rings, and each adds up a channel tile.)
    if (kMode == kWhole) {
      float4* mine = reinterpret_cast<float4*>(stages) + lane;
#pragma unroll
      for (int nq = 0; nq < kNQ; ++nq) {
        mine[(kNQ * kDM + nq) * 32] = make_float4(m[nq][0], l[nq][0], m[nq][1], l[nq][1]);
#pragma unroll
        for (int j = 0; j < kDM; ++j) mine[(nq * kDM + j) * 32] = make_float4(o[nq][j][0], o[nq][j][1], o[nq][j][2], o[nq][j][3]);
      }
      __syncthreads();
      if (warp >= kDM) break;
      const float4* all = reinterpret_cast<const float4*>(smem) + lane;
      constexpr int kStep = G::kWarpBytes / 16;
#pragma unroll
      for (int nq = 0; nq < kNQ; ++nq) {
        float4 ml[kWarps];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) ml[w] = all[w * kStep + (kNQ * kDM + nq) * 32];
        float top[2] = {-INFINITY, -INFINITY}, sum_l[2] = {}, sum_o[4] = {};
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top[0] = fmaxf(top[0], ml[w].x), top[1] = fmaxf(top[1], ml[w].z);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float4 t = all[w * kStep + (nq * kDM + warp) * 32];
          const float f0 = ml[w].x == -INFINITY ? 1.f : ex2_approx(ml[w].x - top[0]);  // (as below)
          const float f1 = ml[w].z == -INFINITY ? 1.f : ex2_approx(ml[w].z - top[1]);
          sum_l[0] += ml[w].y * f0, sum_l[1] += ml[w].w * f1;
          sum_o[0] += t.x * f0, sum_o[1] += t.y * f1, sum_o[2] += t.z * f0, sum_o[3] += t.w * f1;
        }
        const int row = row_base + 8 * nq + g, t = row / p.group;
        __nv_bfloat16* row_out = nullptr;
        if (row < p.rows) row_out = a.out + (((int64_t)b * a.new_tokens + t) * a.hq + h * p.group + row - t * p.group) * a.d;
        float inv[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          inv[x] = sum_l[x] == 0.f ? 0.f : 1.f / sum_l[x];
          const int r = row_base + 8 * nq + 2 * c + x, rt = r / p.group;
          if (warp == 0 && g == 0 && r < p.rows && a.lse)
            a.lse[((int64_t)b * a.new_tokens + rt) * a.hq + h * p.group + r - rt * p.group] = lse_of(top[x], sum_l[x], kFp8 ? kWeightShift : 0.f);
        }
        write_tile<kFp8, kDP>(sum_o, warp, inv, row_out, a.d);
      }
      break;
    }
    if (kMode != kSolo) {
      if (warp > 0) sm100::named_bar(warp, 64);
      else if (pieces > 0) sm100::named_bar(kWarps, 64);
    }
    const bool mine_any = i_begin < i_end, sum_any = kMode != kSolo && warp > 0 && s_any;
    if (sum_any) {
#pragma unroll
      for (int nq = 0; nq < kNQ; ++nq) {
        const float4 ml = s_ml[nq * 32];
        float f[2], fs[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float mo = x ? ml.z : ml.x, lo2 = x ? ml.w : ml.y;
          const float top = fmaxf(m[nq][x], mo);
          // (a maximum of -inf: no key, or no number; what is added is then 0 or not a number)
          f[x] = m[nq][x] == -INFINITY ? 1.f : ex2_approx(m[nq][x] - top);
          fs[x] = mo == -INFINITY ? 1.f : ex2_approx(mo - top);
          m[nq][x] = top;
          l[nq][x] = l[nq][x] * f[x] + lo2 * fs[x];
        }
#pragma unroll
        for (int j = 0; j < kDM; ++j) {
          const float4 t = s_sum[(nq * kDM + j) * 32];
          const float tv[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) o[nq][j][e] = o[nq][j][e] * f[e & 1] + tv[e] * fs[e & 1];
        }
      }
    }
    __syncwarp();  // the sum has been read
    if (kMode != kSolo && warp < kWarps - 1) {
      if (mine_any || warp == 0) {
#pragma unroll
        for (int nq = 0; nq < kNQ; ++nq) {
          s_ml[nq * 32] = make_float4(m[nq][0], l[nq][0], m[nq][1], l[nq][1]);
#pragma unroll
          for (int j = 0; j < kDM; ++j) s_sum[(nq * kDM + j) * 32] = make_float4(o[nq][j][0], o[nq][j][1], o[nq][j][2], o[nq][j][3]);
        }
        if (lane == 0) s_any = mine_any || sum_any;
      }
      __syncwarp();
      sm100::named_bar_arrive(warp + 1, 64);
    } else {
      if (kMode != kSolo && more) sm100::named_bar_arrive(kWarps, 64);
      const int64_t slot = 2 * share + (pieces == 0 ? 0 : 1);
      if (blk == 0 && take == n_blk) {
#pragma unroll
        for (int nq = 0; nq < kNQ; ++nq) {
          const int row = row_base + 8 * nq + g, t = row / p.group;
          __nv_bfloat16* row_out = nullptr;
          if (row < p.rows) row_out = a.out + (((int64_t)b * a.new_tokens + t) * a.hq + h * p.group + row - t * p.group) * a.d;
          float inv[2];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            inv[x] = l[nq][x] == 0.f ? 0.f : 1.f / l[nq][x];
            const int r = row_base + 8 * nq + 2 * c + x, rt = r / p.group;
            if (g == 0 && r < p.rows && a.lse)
              a.lse[((int64_t)b * a.new_tokens + rt) * a.hq + h * p.group + r - rt * p.group] = lse_of(m[nq][x], l[nq][x], kFp8 ? kWeightShift : 0.f);
          }
#pragma unroll
          for (int j = 0; j < kDM; ++j) write_tile<kFp8, kDP>(o[nq][j], j, inv, row_out, a.d);
        }
      } else {
#pragma unroll
        for (int nq = 0; nq < kNQ; ++nq) {
          if (row_base + 8 * nq >= p.rows) continue;
          p.part_ml[(slot * kNQ + nq) * 32 + lane] = make_float4(m[nq][0], l[nq][0], m[nq][1], l[nq][1]);
#pragma unroll
          for (int j = 0; j < kDM; ++j)
            p.part_o[((slot * kNQ + nq) * kDM + j) * 32 + lane] = make_float4(o[nq][j][0], o[nq][j][1], o[nq][j][2], o[nq][j][3]);
        }
      }
    }
    ++pieces;
    slot_out = slot_out == kPlaces - 1 ? 0 : slot_out + 1;
  }
}

// Joins the partial results of every unit that more than one share has a part of, in the order of its
// keys; fp32 sums.  The launch's blocks take jobs in turn: a row tile, its channel tiles a warp each, where a unit
// has few partials; a row tile's one channel tile, the partials dealt to the eight warps, where it
// has many.  (It does not release the launch after it early: CTAs of a next main kernel that are placed
// beside this one's lie unevenly over the SMs.  48 sequences to 8192, three CTAs per SM: 42.4 us a call
// in a row, against 33.4.)
constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32;
constexpr int kFewPartials = 8;
constexpr int kJoinCtas = 3;  // per SM (8 sequences to 131072: 174 us, with two and more registers 177, with four, which spills, 176)

template <bool kFp8, int kDP, int kNQ, Mode kMode>
__global__ void __launch_bounds__(kJoinThreads, kJoinCtas) attn_join_kernel(const __grid_constant__ DecodeParams p, int grid) {
  using G = Geo<kFp8, kDP, kNQ, kMode>;
  constexpr int kDM = kDP / 16, kMost = G::kMaxCtas * G::kShares, kPer = (kMost + kJoinThreads - 1) / kJoinThreads;
  const AttnDecodeArgs& a = p.a;
  __shared__ int s_end[kMost];    // jobs up to and with the unit that share i ends
  __shared__ int4 s_meta[kMost];  // that unit: first partial, partials, unit
  __shared__ int s_warp[kJoinWarps];
  __shared__ int64_t s_sum[kJoinThreads];
  __shared__ float4 s_o[kJoinWarps][32], s_ml[kJoinWarps][32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;

  // Who worked on what follows from the lengths, as in the main kernel (which has begun, so what wrote
  // them is done): found before the wait for its results.
  const int64_t units_per_seq = (int64_t)a.hkv * p.row_blocks;
  const int per = (a.batch + kJoinThreads - 1) / kJoinThreads;
  auto seq_cost = [&](int b, int& n_blk) {
    int lo, hi;
    key_range(a, a.seq_lens[b], lo, hi, nullptr);
    n_blk = num_blocks<G::kBlockTok>(lo, hi);
    return (n_blk + kUnitCost) * units_per_seq;
  };
  int n_blk;
  int64_t mine = 0;
  for (int b = tid * per; b < min(a.batch, (tid + 1) * per); ++b) mine += seq_cost(b, n_blk);
  int64_t incl64 = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t t = __shfl_up_sync(0xffffffffu, incl64, o);
    if (lane >= o) incl64 += t;
  }
  __shared__ int64_t s_wsum[kJoinWarps];
  if (lane == 31) s_wsum[warp] = incl64;
  __syncthreads();
  int64_t cost = 0;
  for (int w = 0; w < kJoinWarps; ++w) {
    if (w < warp) incl64 += s_wsum[w];
    cost += s_wsum[w];
  }
  s_sum[tid] = incl64;  // the cost up to and with this thread's sequences
  __syncthreads();
  const int shares = (int)min(cost, (int64_t)grid * G::kShares);
  auto row_tiles = [&](int unit) { return min(kNQ, (p.rows - (unit % p.row_blocks) * 8 * kNQ + 7) / 8); };
  int jobs = 0;
#pragma unroll 1
  for (int k = 0; k < kPer; ++k) {
    const int i = kPer * tid + k;
    if (i >= shares) break;
    // share i ends a unit that others began if it begins inside that unit's blocks and goes on to their end
    const int64_t w0 = divide(i * cost, shares), w1 = divide((i + 1) * cost, shares);
    int lo = 0, hi = kJoinThreads - 1;  // the first thread whose sum is beyond w0
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (s_sum[mid] > w0) hi = mid;
      else lo = mid + 1;
    }
    int64_t at = lo > 0 ? s_sum[lo - 1] : 0;
    int b = lo * per;
    for (;; ++b) {
      const int64_t n = seq_cost(b, n_blk);
      if (w0 < at + n || b + 1 >= a.batch) break;
      at += n;
    }
    const int n_cost = n_blk + kUnitCost;
    const int u = (int)divide(w0 - at, n_cost), blk = (int)(w0 - at - (int64_t)u * n_cost);
    int4 mt = make_int4(0, 0, 0, 0);
    if (blk > 0 && blk < n_blk && w1 - w0 >= n_blk - blk) {
      // the share with the unit's first block; the unit is its first one if the share begins there, or in
      // the end (without blocks) of the unit before
      const int64_t start = w0 - blk;
      const int64_t c0 = divide((start + 1) * shares - 1, cost);
      mt = make_int4((int)(2 * c0 + (start - divide(c0 * cost, shares) <= kUnitCost ? 0 : 1)), (int)(i - c0 + 1),
                     (int)((int64_t)b * units_per_seq + u), 0);
      jobs += row_tiles(mt.z) * (mt.y > kFewPartials ? kDM : 1);
    }
    s_meta[i] = mt;
    s_end[i] = jobs;  // (of this thread's shares so far)
  }
  int incl = jobs;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += t;
  }
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  int before = 0, total = 0;
  for (int w = 0; w < kJoinWarps; ++w) {
    if (w < warp) before += s_warp[w];
    total += s_warp[w];
  }
  for (int k = 0; k < kPer; ++k)
    if (kPer * tid + k < shares) s_end[kPer * tid + k] += before + incl - jobs;
  __syncthreads();
  // A job: its unit's partials, row tile and channel tile, and where the results go.
  int4 mt = make_int4(0, 0, 0, 0);
  bool many = false;
  int nq = 0, jj = 0;
  int64_t out_g = 0, out_c[2] = {0, 0};  // the token's row of tile rows g and 2 c + {0, 1}; -1 beyond the unit's
  auto find = [&](int job) {
    int lo = 0, hi = shares - 1;  // the first share whose end is beyond the job
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (s_end[mid] > job) hi = mid;
      else lo = mid + 1;
    }
    mt = s_meta[lo];
    const int local = job - (lo > 0 ? s_end[lo - 1] : 0);
    many = mt.y > kFewPartials;
    nq = many ? local / kDM : local;
    jj = many ? local % kDM : warp;
    const int bh = mt.z / p.row_blocks, row_base = (mt.z - bh * p.row_blocks) * 8 * kNQ + 8 * nq;
    const int b = bh / a.hkv, h = bh - b * a.hkv;
    auto row_at = [&](int row) {
      const int t = row / p.group;
      return row < p.rows ? ((int64_t)b * a.new_tokens + t) * a.hq + h * p.group + row - t * p.group : -1;
    };
    out_g = row_at(row_base + g);
    out_c[0] = row_at(row_base + 2 * c);
    out_c[1] = row_at(row_base + 2 * c + 1);
  };
  // (the first one is found before the wait)
  int job = blockIdx.x;
  if (job < total) find(job);
  sm100::griddep_wait();

  for (; job < total; job += gridDim.x) {
    if (job != blockIdx.x) find(job);
    const int share0 = mt.x >> 1;
    auto slot = [&](int i) { return (int64_t)(i == 0 ? mt.x : 2 * (share0 + i)) * kNQ + nq; };
    // partials first, first + step, ..: their results relative to the largest reference met so far
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, o[4] = {0.f, 0.f, 0.f, 0.f};
    auto add = [&](const float4& ml, const float4& t) {
      const float mo[2] = {ml.x, ml.z}, lo2[2] = {ml.y, ml.w}, tv[4] = {t.x, t.y, t.z, t.w};
      float f[2], fs[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float top = fmaxf(m[x], mo[x]);
        f[x] = m[x] == -INFINITY ? 1.f : ex2_approx(m[x] - top);
        fs[x] = mo[x] == -INFINITY ? 1.f : ex2_approx(mo[x] - top);
        m[x] = top;
        l[x] = l[x] * f[x] + lo2[x] * fs[x];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = o[e] * f[e & 1] + tv[e] * fs[e & 1];
    };
    if (jj < kDM) {
      constexpr int kBatch = 4;  // loads under way
      const int step = many ? kJoinWarps : 1;
      for (int i0 = many ? warp : 0; i0 < mt.y; i0 += kBatch * step) {
        float4 ml[kBatch], t[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          const int i = i0 + k * step;
          if (i < mt.y) {
            const int64_t sl = slot(i);
            ml[k] = p.part_ml[sl * 32 + lane];
            t[k] = p.part_o[(sl * kDM + jj) * 32 + lane];
          }
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
          if (i0 + k * step < mt.y) add(ml[k], t[k]);
      }
    }
    if (many) {
      __syncthreads();
      s_o[warp][lane] = make_float4(o[0], o[1], o[2], o[3]);
      s_ml[warp][lane] = make_float4(m[0], l[0], m[1], l[1]);
      __syncthreads();
      if (warp != 0) continue;
      for (int w = 1; w < kJoinWarps; ++w) add(s_ml[w][lane], s_o[w][lane]);
    }
    if (jj < kDM) {
      float inv[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        inv[x] = l[x] == 0.f ? 0.f : 1.f / l[x];
        if (jj == 0 && g == 0 && out_c[x] >= 0 && a.lse) a.lse[out_c[x]] = lse_of(m[x], l[x], kFp8 ? kWeightShift : 0.f);
      }
      write_tile<kFp8, kDP>(o, jj, inv, out_g >= 0 ? a.out + out_g * a.d : nullptr, a.d);
    }
  }
}

// Row tiles of one unit: 1 up to 8 rows of a (sequence, kv head), else 2, and as many units as the rows
// need.  (Units of 4 tiles read a long cache once for 32 rows, but took as long per row there, and up to
// 1.6 times as long for short sequences: 851 against 555 us for 80 rows of 208 x 402 tokens.)
int row_tiles(int rows) { return rows <= 8 ? 1 : 2; }
int padded_dim(int d) { return d <= 64 ? 64 : 128; }

template <bool kFp8, int kDP, int kNQ, Mode kMode>
cudaError_t launch_typed(const AttnDecodeArgs& a, cudaStream_t stream) {
  using G = Geo<kFp8, kDP, kNQ, kMode>;
  using SM = Smem<kFp8, kDP, kNQ, kMode>;
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
  int64_t grid = (int64_t)G::kCtas * sms;
  if (grid > G::kMaxCtas) grid = G::kMaxCtas;
  const int64_t most_shares = units < grid * G::kWarps ? units * (most_blocks + kUnitCost) : INT64_MAX;
  if (most_shares < grid * G::kShares) grid = (most_shares + G::kShares - 1) / G::kShares;
  if (kMode == kWhole) grid = units;
  uint8_t* ws = a.workspace;
  p.status = reinterpret_cast<uint32_t*>(ws);
  p.part_ml = reinterpret_cast<float4*>(ws + kWorkspaceHeader);
  p.part_o = p.part_ml + 2 * kMaxShares * kNQ * 32;
  constexpr uint32_t kSmem = SM::kTotal + 128;
  cudaError_t e = set_smem_once(attn_decode_kernel<kFp8, kDP, kNQ, kMode>, kSmem, attr_done);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(G::kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, attn_decode_kernel<kFp8, kDP, kNQ, kMode>, p);
  if constexpr (kMode != kWhole) {
    if (e != cudaSuccess || most_blocks == 1) return e;  // (no unit is in two shares: nothing to join)
    cfg.gridDim = dim3((unsigned)(kJoinCtas * sms));
    cfg.blockDim = dim3(kJoinThreads);
    cfg.dynamicSmemBytes = 0;
    e = cudaLaunchKernelEx(&cfg, attn_join_kernel<kFp8, kDP, kNQ, kMode>, p, (int)grid);
  }
  return e;
}

// Units per warp from which warps take shares of their own: their results of a unit need no joining
// then, but a unit is one warp's work.  (128 sequences, 8 kv heads, bf16: 80 rows, 5120 units, take 149 us
// in common and 77 alone at 120 keys, 466 and 439 at 2000; 16 rows, 1024 units, 35 and 41, 105 and 124.)
constexpr int64_t kSoloUnits = 4;
// Keys in the tables (or the window) up to which units that all find an SM are not split: one launch,
// no join, but a unit is one CTA's work.  The more units there are, the less splitting them helps;
// lengths that differ are what the second bound is for.  (bf16, 4 rows of 128 channels, split and whole:
// 8 units take 10.1 and 6.8 us at 333 keys, 10.2 and 9.4 at 760, 11.2 and 14.3 at 1500; 128 units 14.0 and
// 7.4, 16.9 and 10.1, 18.3 and 14.7.  16 rows, 8 units: 12.7 and 9.4, 11.5 and 13.2.)
constexpr int64_t kWholeKeys = 640, kWholeMost = 1024;

template <bool kFp8, int kDP, int kNQ>
cudaError_t launch_mode(const AttnDecodeArgs& a, int64_t units, cudaStream_t stream) {
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  if (units >= kSoloUnits * Geo<kFp8, kDP, kNQ, kSolo>::kWarps * Geo<kFp8, kDP, kNQ, kSolo>::kCtas * sms) return launch_typed<kFp8, kDP, kNQ, kSolo>(a, stream);
  int64_t keys = (int64_t)a.max_pages << a.page_shift;  // the most that a unit can have
  if (a.window > 0) keys = std::min<int64_t>(keys, (int64_t)a.window + a.new_tokens - 1);
  if (units <= sms && keys <= kWholeMost && keys * (sms - units) <= kWholeKeys * sms)
    return launch_typed<kFp8, kDP, kNQ, kWhole>(a, stream);
  return launch_typed<kFp8, kDP, kNQ, kCommon>(a, stream);
}

template <bool kFp8, int kDP>
cudaError_t launch_rows(const AttnDecodeArgs& a, cudaStream_t stream) {
  const int rows = a.new_tokens * (a.hq / a.hkv), tiles = row_tiles(rows);
  const int64_t units = (int64_t)a.batch * a.hkv * ((rows + 8 * tiles - 1) / (8 * tiles));
  return tiles == 2 ? launch_mode<kFp8, kDP, 2>(a, units, stream) : launch_mode<kFp8, kDP, 1>(a, units, stream);
}

}  // namespace

size_t attn_decode_workspace_bytes(int32_t rows, int32_t d) {
  const size_t tiles = row_tiles(rows);
  return kWorkspaceHeader + 2 * (size_t)kMaxShares * tiles * 32 * sizeof(float4) * (1 + padded_dim(d) / 16);
}

cudaError_t launch_attn_decode(const AttnDecodeArgs& a, cudaStream_t stream) {
  if ((int64_t)a.batch * a.new_tokens == 0) return cudaSuccess;
  if (a.k_scale) return a.d <= 64 ? launch_rows<true, 64>(a, stream) : launch_rows<true, 128>(a, stream);
  return a.d <= 64 ? launch_rows<false, 64>(a, stream) : launch_rows<false, 128>(a, stream);
}

}  // namespace kda
