// paged_attn_decode_sparse: one query token per sequence attending to the
// selected blocks of its KV head,
//     s_j = scale * q.k_j + slope_h * (j - i),   out = softmax(s) . V
// over the keys j of the selected blocks with j <= i = L - 1 inside the
// sliding window.
//
// Bound by reading the selected keys and values (2 D elements per key and KV
// head).  A group's query heads are rows of one m16 tile of mma.sync, so they
// share every byte of K and V; tcgen05's smallest tile, 64 rows, would be
// mostly empty.  CTA = (part of the selection, KV head x 16 rows, sequence), 3 to
// 8 warps, each walking its own 16-key units (a block is one or two) through a
// two-stage ring of TMA boxes (16 keys x 64 channels, 128-byte swizzle; K and
// V), one pass with the running maximum (moved, and the output rescaled, only
// when a score passes it by 2^8) and sum of the softmax.  The lane that will
// need it loads a unit's block number and place, 32 units of a warp at a time,
// so there is no table in shared memory and no limit to the selection's length.
//
// The parts of one selection are a cluster: their (m, l, O) are joined through
// distributed shared memory, every CTA writing a share of the output.  No
// second kernel, no workspace, and the same order of additions every time.
//
// The tensor map fetches no more of a line than a head's row: with the 256-byte
// promotion of the dense kernels a 128-byte row brought its neighbour's along (32
// sequences, 16 KV heads of 64: 69 against 52 us).  Measured: 64 sequences, 128
// blocks of 16 for each of 8 KV heads of 128, 538 MB in 89 us (6.1 TB/s).
//
// Over an fp8 cache the boxes carry the codes.  q.k runs on them as they are:
// each query row scaled by a power of two of its own and split into two E4M3
// terms for bf16, three for fp16 (4 bits each: the 8 and 11 bits of a component,
// exact within 2^9 and 2^6 of the row's largest and off by 2^-17 of it below); with
// four rows or fewer the first two in one product, the low ones as rows 4 .. 7.  The
// channels are taken in an order in which a lane's 16-byte chunk of a key is its
// own fragment.  p.V runs transposed on fp16 operands: the weights' fragments
// are the B operand, V^T is built from the codes by byte permutes.
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "mma.cuh"

namespace pkv {
namespace sparse {

constexpr int kUnit = 16;    // keys per unit (one TMA box height)
constexpr int kRows = 16;    // query heads per CTA: one m16 tile
constexpr int kStages = 2;   // of a warp's ring
constexpr int kMaxParts = 8;  // CTAs of a cluster
constexpr float kLazy = 8.f;
constexpr int kFar = 0x7fffffe0;  // "position" of a unit that nothing may read
constexpr float kLowest = -3.4028234663852886e38f;

struct Args {
  void *out;
  const uint16_t *query;
  const int32_t *block_tables, *seq_lens, *selected;
  const float *alibi;
  int64_t num_blocks;
  int max_blocks_per_seq, max_selected, H, KVH, QPK, BS, window;
  int row_groups, parts;
  float scale_log2, v_scale;
};

template <int D, bool KV8, int W>
struct Lay {
  static constexpr int BOX = kUnit * 128;     // 16 rows x 64 channels x 2 B
  static constexpr int V16 = (D / 64) * BOX;  // one unit of K or V as 16-bit values
  static constexpr int TILE = KV8 ? kUnit * D : V16;
  static constexpr int STAGE = 2 * TILE;
  // the warps' rings, then (16-bit cache) a zero V tile; the merge reuses it
  static constexpr int ZERO = W * kStages * STAGE;
  static constexpr int PAD = D + 8;  // floats of a row of the merge: no bank conflicts
  static constexpr int MERGE = (W + 1) * kRows * (PAD + 2) * 4;
  static constexpr int RING = ZERO + (KV8 ? 0 : V16);
  static constexpr int SMEM = 1024 + (RING > MERGE ? RING : MERGE);
};

// Byte offset of 16-byte chunk `chunk` (8 channels) of key row `tok` in a
// 16-bit tile: 64-channel box, row, 128-byte swizzle.
__device__ __forceinline__ uint32_t swz16(int tok, int chunk) {
  return static_cast<uint32_t>((chunk >> 3) * (kUnit * 128) + tok * 128 +
                               (((chunk & 7) ^ (tok & 7)) << 4));
}
// The same in a tile of codes (D bytes a row; 128- or 64-byte swizzle).
template <int D>
__device__ __forceinline__ uint32_t swz8(int row, int chunk) {
  if constexpr (D == 128)
    return static_cast<uint32_t>(row * 128 + ((chunk ^ (row & 7)) << 4));
  else
    return static_cast<uint32_t>(row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4));
}
__device__ __forceinline__ uint32_t word_of(const uint4 &v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}
// Bytes {a[j], b[j], a[j+1], b[j+1]}, j = 0 or 2.
__device__ __forceinline__ uint32_t interleave2(uint32_t a, uint32_t b, int j) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(j ? 0x7362u : 0x5140u));
  return r;
}

// Warps of a CTA: kFew for grids of less than a CTA per SM, else as many as
// let four to five CTAs share an SM (their copies go on while one starts or
// joins).
constexpr int kFew = 8;
template <int D, bool KV8>
constexpr int kMany = D == 128 && !KV8 ? 3 : 4;
// E4M3 codes of what two terms leave of four values.
__device__ __forceinline__ uint32_t rest_e4m3x4(const float *v, uint32_t hi, uint32_t lo) {
  const uint2 a = e4m3x4_to_h4(hi), b = e4m3x4_to_h4(lo);
  const float2 a0 = FP16::to_f2(a.x), a1 = FP16::to_f2(a.y);
  const float2 b0 = FP16::to_f2(b.x), b1 = FP16::to_f2(b.y);
  uint32_t c, none;
  split_e4m3x4(v[0] - a0.x - b0.x, v[1] - a0.y - b0.y, v[2] - a1.x - b1.x, v[3] - a1.y - b1.y, c,
               none);
  return c;
}

// The leading 8 or 11 bits of x: a bf16 value, an fp16 value in its normal range.
__device__ __forceinline__ float leading(float x, BF16) {
  return __uint_as_float(__float_as_uint(x) & 0xffff0000u);
}
__device__ __forceinline__ float leading(float x, FP16) {
  return __uint_as_float(__float_as_uint(x) & 0xffffe000u);
}
// A pair of values >= 0 with zeros replaced: by bf16's 2^-126, by fp16's 2^-24.
__device__ __forceinline__ uint32_t above_zero(uint32_t w, BF16) {
  uint32_t d;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(w), "r"(0x00800080u));
  return d;
}
__device__ __forceinline__ uint32_t above_zero(uint32_t w, FP16) {
  uint32_t d;
  asm("max.f16x2 %0, %1, %2;" : "=r"(d) : "r"(w), "r"(0x00010001u));
  return d;
}

// A row's output: zero where no key was visible, NaN where all scores were -infinity.
__device__ __forceinline__ float joined(float m, float num, float den) {
  return m == -INFINITY ? 0.f : den == 0.f ? NAN : num / den;
}

// CTAs per SM that registers are kept for (shared memory allows as many).  One
// fewer for 8 rows of bf16 over an fp8 cache, which would spill (256 sequences,
// 8 KV heads of 128: 149 / 157 us; of 64: 90 / 93; fp16, whose third query term
// spills either way, 182 / 171).
template <class T, int D, bool KV8, int ROWS, int W>
constexpr int kCtasPerSm =
    W == kFew ? 1
              : (D == 64 ? (ROWS > 8 ? 4 : 5) : KV8 && ROWS > 8 ? 3 : 4) -
                    (KV8 && ROWS == 8 && std::is_same<T, BF16>::value ? 1 : 0);

// ROWS: 16, or 8 for groups of no more query heads (rows 8 .. 15 of the tile are
// not kept), or over an fp8 cache 4 (rows 4 .. 7 are the low terms of 0 .. 3).
template <class T, int D, bool KV8, int ROWS, int W>
__global__ void __launch_bounds__(32 * W, kCtasPerSm<T, D, KV8, ROWS, W>)
sparse_kernel(const Args a, const __grid_constant__ CUtensorMap tmap) {
  constexpr int kWarps = W, kThreads = 32 * W;
  using L_ = Lay<D, KV8, W>;
  using MT = std::conditional_t<KV8, FP16, T>;  // type of the weights and of V
  constexpr bool HALF = ROWS <= 8, fold = ROWS == 4;
  static_assert(KV8 || !fold, "a 16-bit tile's low terms are in rows 8 .. 15");
  constexpr int NR = HALF ? 1 : 2;              // row halves a lane keeps (g, g + 8)
  constexpr int KS = D / 16, NT = D / 8, KS8 = D / 32;
  // fp16 weights of a 16-bit cache are 2^6 times e^(s - m), 2^14 at most: what takes
  // the place of a zero low term is 2^-30 of the largest
  constexpr float kLift = !KV8 && std::is_same<T, FP16>::value ? 6.f : 0.f;
  constexpr bool kThird = KV8 && std::is_same<T, FP16>::value;  // a third query term
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  __shared__ uint64_t bars[kWarps][kStages];
  __shared__ int spos[kWarps][kStages];  // position of a stage's first key
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = blockIdx.x;
  const int kvh = blockIdx.y / a.row_groups, rg = blockIdx.y % a.row_groups;
  const int b = blockIdx.z;
  if (threadIdx.x == 0) prefetch_tensormap(&tmap);
  uint64_t *wbar = bars[warp];
  if (lane == 0) {
    for (int st = 0; st < kStages; ++st) mbar_init(&wbar[st], 1);
    fence_mbar_init();
  }
  if constexpr (!KV8)
    for (int i = threadIdx.x; i < L_::V16 / 16; i += kThreads)
      reinterpret_cast<uint4 *>(smem + L_::ZERO)[i] = make_uint4(0u, 0u, 0u, 0u);
  __syncthreads();
  grid_dependency_wait();
  grid_launch_dependents();

  int L = __ldg(a.seq_lens + b);
  if (L < 0 || L > static_cast<int64_t>(a.max_blocks_per_seq) * a.BS) {
    if (part == 0 && blockIdx.y == 0 && threadIdx.x == 0) record_error(PKV_ERR_BOUNDS, b);
    L = 0;
  }
  const int i_pos = L - 1, lo = a.window > 0 ? max(0, L - a.window) : 0;
  const int nblk = (L + a.BS - 1) / a.BS;

  // ---- this part of the selection's places, as 16-key units ------------------------
  const int64_t sel0 = (static_cast<int64_t>(b) * a.KVH + kvh) * a.max_selected;
  const int32_t *sel = a.selected + sel0;
  const int32_t *table = a.block_tables + static_cast<int64_t>(b) * a.max_blocks_per_seq;
  const int upb = a.BS / kUnit;
  // a valid selection is no longer than the sequence has blocks; behind that only
  // negative numbers may stand, which are looked at below and not shared out
  const int n_places = min(a.max_selected, nblk);
  const int units = n_places * upb;
  const int per = (units + a.parts - 1) / a.parts;
  const int u_begin = min(part * per, units), nu = min(per, units - u_begin);
  const int places = nu > warp ? (nu - warp + kWarps - 1) / kWarps : 0;

  // unit i of this warp: cache row and position of its first key (row -1: no
  // block is selected there)
  auto place = [&](int i, int &row, int &pos) {
    row = -1;
    pos = kFar;
    if (i >= places) return;
    const int u = u_begin + warp + i * kWarps, e = u / upb;
    const int s = __ldg(sel + e), prev = e ? __ldg(sel + e - 1) : -1;
    if (s < 0 || L == 0) return;
    row = 0;
    if (s >= nblk || (e && (prev < 0 || prev >= s))) {
      record_error(PKV_ERR_BOUNDS, sel0 + e);
      return;
    }
    const int pb = __ldg(table + s);
    if (pb < 0 || pb >= a.num_blocks) {
      record_error(PKV_ERR_BOUNDS, static_cast<int64_t>(b) * a.max_blocks_per_seq + s);
      return;
    }
    row = pb * a.BS + (u % upb) * kUnit;
    pos = s * a.BS + (u % upb) * kUnit;
  };
  // this lane's unit of the 32 being issued and of the next 32, and which of
  // the former are still to come
  int row_c, pos_c, row_n, pos_n, base = 0;
  place(lane, row_c, pos_c);
  place(32 + lane, row_n, pos_n);
  uint32_t left = __ballot_sync(0xffffffffu, row_c >= 0);
  uint8_t *wt = smem + warp * kStages * L_::STAGE;
  int issued = 0;
  auto issue = [&]() {  // by the whole warp: the next unit's copies, if there is one
    while (left == 0 && base + 32 < places) {
      base += 32;
      row_c = row_n;
      pos_c = pos_n;
      place(base + 32 + lane, row_n, pos_n);
      left = __ballot_sync(0xffffffffu, row_c >= 0);
    }
    if (left == 0) return;
    const int k = issued++, from = __ffs(left) - 1;
    left &= left - 1;
    const int row = __shfl_sync(0xffffffffu, row_c, from);
    const int pos = __shfl_sync(0xffffffffu, pos_c, from);
    if (lane == 0) {
      const int st = k % kStages;
      spos[warp][st] = pos;
      mbar_arrive_expect_tx(&wbar[st], 2u * L_::TILE);
      uint8_t *kt = wt + st * L_::STAGE;
      if constexpr (KV8) {
        tma_load_4d(kt, &tmap, &wbar[st], 0, kvh, row, 0);
        tma_load_4d(kt + L_::TILE, &tmap, &wbar[st], 0, kvh, row, 1);
      } else {
#pragma unroll
        for (int r = 0; r < D / 64; ++r) {
          tma_load_4d(kt + r * L_::BOX, &tmap, &wbar[st], 64 * r, kvh, row, 0);
          tma_load_4d(kt + L_::TILE + r * L_::BOX, &tmap, &wbar[st], 64 * r, kvh, row, 1);
        }
      }
    }
  };
  for (int st = 0; st < kStages; ++st) issue();
  if (L > 0)
    for (int e = n_places + part * kThreads + threadIdx.x; e < a.max_selected;
         e += a.parts * kThreads)
      if (__ldg(sel + e) >= 0) record_error(PKV_ERR_BOUNDS, sel0 + e);

  // ---- query fragments -----------------------------------------------------------
  const int g = lane >> 2, tq = lane & 3;
  bool valid[2];
  int head[2];
  float slope[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int r = rg * kRows + g + 8 * x;
    valid[x] = x < NR && r < a.QPK;
    head[x] = kvh * a.QPK + (valid[x] ? r : 0);
    slope[x] = a.alibi && valid[x] ? __ldg(a.alibi + head[x]) * kLog2e : 0.f;
    if (x == 0 && fold && a.alibi) {  // rows 4 .. 7 weigh as rows 0 .. 3 do
      const int rs = min(g & 3, a.QPK - 1);
      slope[0] = __ldg(a.alibi + kvh * a.QPK + rs) * kLog2e;
    }
  }
  const uint16_t *qb = a.query + static_cast<int64_t>(b) * a.H * D;
  uint32_t qa[KS][4], qc[kThird ? KS8 : 1][4];
  float sl2[2] = {a.scale_log2, a.scale_log2};  // of rows g, g + 8
  if constexpr (KV8) {
    // qa[s] = high, qa[KS8 + s] = low terms of k-step s: this lane's channels
    // tq * D / 4 + 8 s .. + 7
    const int srow = rg * kRows + (fold ? (g & 3) : g);
    const bool src_valid = srow < a.QPK;
    const int src_head = kvh * a.QPK + (src_valid ? srow : 0);
    auto chunk = [&](int x, int s) -> uint4 {
      const int h = x == 0 ? src_head : head[1];
      const bool v = x == 0 ? src_valid : valid[1];
      const uint4 *p = reinterpret_cast<const uint4 *>(qb + h * D + tq * (D / 4));
      return v ? __ldg(p + s) : make_uint4(0u, 0u, 0u, 0u);
    };
    // each row by its own power of two: largest finite |q| * 2^-e in [2^7, 2^8)
    float mul[NR];
#pragma unroll
    for (int x = 0; x < NR; ++x) {
      uint32_t am = 0;  // its largest finite |q|, as bits
#pragma unroll
      for (int s = 0; s < KS8; ++s) {
        const uint4 u = chunk(x, s);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 f = T::to_f2(word_of(u, k));
          am = max(am, max(finite_bits(f.x), finite_bits(f.y)));
        }
      }
      // (the row's other channels are in the quad's other lanes)
      am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
      am = max(am, __shfl_xor_sync(0xffffffffu, am, 2));
      const int E = static_cast<int>(am >> 23);
      const int e = E == 0 ? 0 : max(-126, E - 134);  // 2^-e and 2^e are normal: e <= 120
      mul[x] = __int_as_float((127 - e) << 23);
      sl2[x] *= __int_as_float((127 + e) << 23);
    }
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int c = 0; c < 4; ++c) qa[s][c] = 0u;
    if constexpr (kThird)
#pragma unroll
      for (int s = 0; s < KS8; ++s)
#pragma unroll
        for (int c = 0; c < 4; ++c) qc[s][c] = 0u;
#pragma unroll
    for (int x = 0; x < NR; ++x)
#pragma unroll
      for (int s = 0; s < KS8; ++s) {
        const uint4 u = chunk(x, s);
        float v[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 f = T::to_f2(word_of(u, k));
          v[2 * k] = scaled_query(f.x, mul[x]);
          v[2 * k + 1] = scaled_query(f.y, mul[x]);
        }
        split_e4m3x4(v[0], v[1], v[2], v[3], qa[s][x], qa[KS8 + s][x]);
        split_e4m3x4(v[4], v[5], v[6], v[7], qa[s][2 + x], qa[KS8 + s][2 + x]);
        if constexpr (kThird) {
          qc[s][x] = rest_e4m3x4(v, qa[s][x], qa[KS8 + s][x]);
          qc[s][2 + x] = rest_e4m3x4(v + 4, qa[s][2 + x], qa[KS8 + s][2 + x]);
          if (x == 0 && fold && g >= 4) qc[s][0] = qc[s][2] = 0u;  // rows 0 .. 3 alone
        }
        if (x == 0 && fold && g >= 4) {  // rows 4 .. 7 hold the low terms
          qa[s][0] = qa[KS8 + s][0];
          qa[s][2] = qa[KS8 + s][2];
        }
      }
  } else {
    const uint32_t *q0 = reinterpret_cast<const uint32_t *>(qb + head[0] * D);
    const uint32_t *q1 = reinterpret_cast<const uint32_t *>(qb + head[1] * D);
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      qa[s][0] = valid[0] ? __ldg(q0 + 8 * s + tq) : 0u;
      qa[s][1] = valid[1] ? __ldg(q1 + 8 * s + tq) : 0u;
      qa[s][2] = valid[0] ? __ldg(q0 + 8 * s + 4 + tq) : 0u;
      qa[s][3] = valid[1] ? __ldg(q1 + 8 * s + 4 + tq) : 0u;
    }
  }

  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  // 16-bit cache: o[n][2 x + c] of row g + 8 x, channels 8 n + 2 tq + c.
  // fp8: the same registers as transposed tiles ot[mt][nt][c]
  float o[NT][2 * NR];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int c = 0; c < 2 * NR; ++c) o[n][c] = 0.f;
  float(&ot)[KS][NR][4] = *reinterpret_cast<float(*)[KS][NR][4]>(&o[0][0]);
  const bool has_alibi = a.alibi != nullptr;
  const int mi = lane >> 3, rr = lane & 7;
  const int k_tok = (mi >> 1) * 8 + rr, k_half = mi & 1;  // ldmatrix rows of K
  const int v_tok = (mi & 1) * 8 + rr, v_half = mi >> 1;  // and of V^T
  bool ok = true;
  bool seen = false;  // a visible key
  int consumed = 0;

  for (int k = 0; k < issued; ++k) {
    const int st = k % kStages;
    const bool got = mbar_wait_bounded(&wbar[st], (k / kStages) & 1, b);
    if (!__all_sync(0xffffffffu, got)) {
      ok = false;
      break;
    }
    consumed = k + 1;
    const uint8_t *tile = wt + st * L_::STAGE;
    const uint32_t kt = smem_u32(tile);
    const int j0 = spos[warp][st];

    // ---- S = Q K^T: two n-tiles of 8 keys, even and odd k-steps apart --------------
    float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    float sd[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    if constexpr (KV8) {
      constexpr int KC = D / 64;
      uint4 kk[2][KC];
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int c = 0; c < KC; ++c)
          kk[n][c] = *reinterpret_cast<const uint4 *>(tile + swz8<D>(g + 8 * n, tq * KC + c));
#pragma unroll
      for (int s = 0; s < KS8; ++s)
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const uint32_t b0 = word_of(kk[n][(2 * s) / 4], (2 * s) % 4);
          const uint32_t b1 = word_of(kk[n][(2 * s + 1) / 4], (2 * s + 1) % 4);
          auto mul = [&](float(&c)[4], const uint32_t(&q)[4]) {
            mma_16832_e4m3(c, q[0], HALF ? 0u : q[1], q[2], HALF ? 0u : q[3], b0, b1, c[0], c[1],
                           HALF ? 0.f : c[2], HALF ? 0.f : c[3]);
          };
          if constexpr (fold) {
            mul((s & 1) ? sd[n] : sc[n], qa[s]);
          } else {
            mul(sc[n], qa[s]);
            mul(sd[n], qa[KS8 + s]);
          }
          if constexpr (kThird) mul((s & 1) ? sc[n] : sd[n], qc[s]);
        }
    } else {
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        uint32_t kb[4];
        ldmatrix_x4(kt + swz16(k_tok, 2 * s + k_half), kb);
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          float(&c)[4] = (s & 1) ? sd[n] : sc[n];
          mma_16816<MT>(c, qa[s][0], HALF ? 0u : qa[s][1], qa[s][2], HALF ? 0u : qa[s][3],
                        kb[2 * n], kb[2 * n + 1], c[0], c[1], HALF ? 0.f : c[2],
                        HALF ? 0.f : c[3]);
        }
      }
    }
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int c = 0; c < 2 * NR; ++c) sc[n][c] += sd[n][c];
    if constexpr (fold) {  // row g + 4 holds row g's low terms
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) sc[n][c] += __shfl_xor_sync(0xffffffffu, sc[n][c], 16);
    }
    // ---- scores in the log2 domain, masked -------------------------------------------
    // sc[n][2 r + c]: row g + 8 r, key j0 + 8 n + 2 tq + c
    const bool interior = j0 >= lo && j0 + kUnit <= L;
    seen |= j0 < L && j0 + kUnit > lo;
    float x[2][4];
    bool grow = false;
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int j = j0 + 8 * n + 2 * tq + c;
          float v = sc[n][2 * r + c] * sl2[r];
          if (has_alibi) v = fmaf(slope[r], static_cast<float>(j - i_pos), v);
          if (!interior && (j < lo || j >= L)) v = -INFINITY;
          x[r][2 * n + c] = v;
          grow |= v > m[r] + kLazy;
        }
    if (__any_sync(0xffffffffu, grow)) {
      float al[2] = {1.f, 1.f};
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        float mx = fmaxf(fmaxf(x[r][0], x[r][1]), fmaxf(x[r][2], x[r][3]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float mn = fmaxf(m[r], mx);
        if (mn > m[r]) {
          al[r] = m[r] == -INFINITY ? 0.f : fast_exp2(m[r] - mn);
          m[r] = mn;
          l[r] *= al[r];
          if constexpr (!KV8) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              o[n][2 * r] *= al[r];
              o[n][2 * r + 1] *= al[r];
            }
          }
        }
      }
      if constexpr (KV8) {
        // O^T's columns are rows 8 nt + 2 tq, + 1, which lanes 8 tq, 8 tq + 4 own
#pragma unroll
        for (int nt = 0; nt < NR; ++nt) {
          const float a0 = __shfl_sync(0xffffffffu, al[nt], 8 * tq);
          const float a1 = __shfl_sync(0xffffffffu, al[nt], 8 * tq + 4);
#pragma unroll
          for (int mt = 0; mt < KS; ++mt) {
            ot[mt][nt][0] *= a0;
            ot[mt][nt][1] *= a1;
            ot[mt][nt][2] *= a0;
            ot[mt][nt][3] *= a1;
          }
        }
      }
    }
    // ---- weights: as two terms of the product's type, p = hi + lo within 2^-16 of it
    // (bf16; fp16 2^-22); their sum l is of the unrounded.  A tile of 8 rows or
    // fewer has the low terms in its other 8 rows (16-bit cache) or, of 4 rows, in
    // rows 4 .. 7 (fp8): no product more.  (One rounded term put up to 2^-8 of a
    // bf16 weight into the output; the second costs 0 to 1% there, and where it is a
    // product of its own 2% of 16 rows over 16 bits and 6 to 9% over fp8.)  Over a
    // 16-bit cache lo is above zero, so that an infinite value stays one: hi is p's
    // leading bits, lo what is left or next to nothing.
    uint32_t pa[4] = {0u, 0u, 0u, 0u}, pl[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const float mr = (m[r] == -INFINITY ? 0.f : m[r]) - kLift;
      float p[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) p[c] = fast_exp2(x[r][c] - mr);
      l[r] += (p[0] + p[1]) + (p[2] + p[3]);
      if constexpr (KV8) {
        pa[r] = MT::from_f2(p[0], p[1]);
        pa[2 + r] = MT::from_f2(p[2], p[3]);
        const float2 h01 = MT::to_f2(pa[r]), h23 = MT::to_f2(pa[2 + r]);
        pl[r] = MT::from_f2(p[0] - h01.x, p[1] - h01.y);
        pl[2 + r] = MT::from_f2(p[2] - h23.x, p[3] - h23.y);
      } else {
        float hi[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) hi[c] = leading(p[c], T{});
        pa[r] = MT::from_f2(hi[0], hi[1]);
        pa[2 + r] = MT::from_f2(hi[2], hi[3]);
        pl[r] = above_zero(MT::from_f2(p[0] - hi[0], p[1] - hi[1]), T{});
        pl[2 + r] = above_zero(MT::from_f2(p[2] - hi[2], p[3] - hi[3]), T{});
      }
    }
    if constexpr (HALF) {
      if constexpr (!KV8) {
        pa[1] = pl[0];
        pa[3] = pl[2];
      } else if (fold && g >= 4) {
        pa[0] = pl[0];
        pa[2] = pl[2];
      }
    }
    // ---- O += P V.  A masked key's V may hold anything, NaN too, and 0 * NaN is
    // NaN: its row is read as zeros.
    if constexpr (KV8) {
      constexpr int VW = D / 32;  // words of this lane's chunk of a key
      const uint8_t *vc = tile + L_::TILE;
      uint32_t vw[4][VW];  // keys 2 tq, 2 tq + 1, 2 tq + 8, 2 tq + 9
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        const int kr = 2 * tq + (kk & 1) + 8 * (kk >> 1);
        if constexpr (D == 128) {
          const uint4 u = *reinterpret_cast<const uint4 *>(vc + swz8<D>(kr, g));
          vw[kk][0] = u.x;
          vw[kk][1] = u.y;
          vw[kk][2] = u.z;
          vw[kk][3] = u.w;
        } else {
          const uint2 u = *reinterpret_cast<const uint2 *>(vc + swz8<D>(kr, g >> 1) + 8 * (g & 1));
          vw[kk][0] = u.x;
          vw[kk][1] = u.y;
        }
        if (!interior && (j0 + kr < lo || j0 + kr >= L)) {
#pragma unroll
          for (int w = 0; w < VW; ++w) vw[kk][w] = 0u;
        }
      }
#pragma unroll
      for (int mt = 0; mt < KS; ++mt) {
        const int w = mt >> 1, j = (mt & 1) * 2;
        const uint2 h01 = e4m3x4_to_h4(interleave2(vw[0][w], vw[1][w], j));
        const uint2 h89 = e4m3x4_to_h4(interleave2(vw[2][w], vw[3][w], j));
#pragma unroll
        for (int nt = 0; nt < NR; ++nt) {
          float(&c)[4] = ot[mt][nt];
          mma_16816<FP16>(c, h01.x, h01.y, h89.x, h89.y, pa[nt], pa[2 + nt], c[0], c[1], c[2],
                          c[3]);
          if constexpr (!fold)
            mma_16816<FP16>(c, h01.x, h01.y, h89.x, h89.y, pl[nt], pl[2 + nt], c[0], c[1], c[2],
                            c[3]);
        }
      }
    } else {
      uint32_t vt = kt + L_::TILE;
      if (!interior && (j0 + v_tok < lo || j0 + v_tok >= L)) vt = smem_u32(smem + L_::ZERO);
#pragma unroll
      for (int n2 = 0; n2 < NT / 2; ++n2) {
        uint32_t vb[4];
        ldmatrix_x4_trans(vt + swz16(v_tok, 2 * n2 + v_half), vb);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float c[4] = {o[2 * n2 + i][0], o[2 * n2 + i][1], 0.f, 0.f};
          if constexpr (!HALF) {
            c[2] = o[2 * n2 + i][2];
            c[3] = o[2 * n2 + i][3];
          }
          mma_16816<MT>(c, pa[0], pa[1], pa[2], pa[3], vb[2 * i], vb[2 * i + 1], c[0], c[1], c[2],
                        c[3]);
          if constexpr (HALF) {
            o[2 * n2 + i][0] = c[0] + c[2];
            o[2 * n2 + i][1] = c[1] + c[3];
          } else {
            mma_16816<MT>(c, pl[0], pl[1], pl[2], pl[3], vb[2 * i], vb[2 * i + 1], c[0], c[1], c[2],
                          c[3]);
#pragma unroll
            for (int x = 0; x < 4; ++x) o[2 * n2 + i][x] = c[x];
          }
        }
      }
    }
    __syncwarp();  // every lane has read the stage: refill it
    issue();
  }
  if (!ok)  // this warp's copies still in flight
    for (int k = consumed; k < issued; ++k)
      mbar_wait_bounded(&wbar[k % kStages], (k / kStages) & 1, b);

  // ---- the warps' (m, l, O) joined, then the cluster's --------------------------------
  // m is -infinity still where no key was visible, and where every score was NaN
  // (l and O are NaN) or -infinity (l is 0): these rows take the lowest finite m, so
  // that they weigh nothing beside a finite score, NaN stays, and a row that had no
  // other has a sum of 0 and is NaN
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    if (seen && m[r] == -INFINITY) m[r] = kLowest;
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
  }
  if constexpr (fold) {  // columns 2 tq + 4, + 5 of O^T hold the low terms' share of 2 tq, + 1
#pragma unroll
    for (int mt = 0; mt < KS; ++mt)
#pragma unroll
      for (int c = 0; c < 4; ++c) ot[mt][0][c] += __shfl_xor_sync(0xffffffffu, ot[mt][0][c], 2);
  }
  __syncthreads();  // all copies have landed: the rings are free
  float *sm = reinterpret_cast<float *>(smem);   // [kWarps + 1][row]: the warps', the CTA's
  float *sl = sm + (kWarps + 1) * kRows;          // [kWarps + 1][row]
  float *so = sl + (kWarps + 1) * kRows;          // [kWarps + 1][row][D]
  if (tq == 0) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      sm[warp * kRows + g + 8 * r] = ok ? m[r] : -INFINITY;
      sl[warp * kRows + g + 8 * r] = ok ? l[r] : 0.f;
    }
  }
  if constexpr (KV8) {
#pragma unroll
    for (int mt = 0; mt < KS; ++mt)
#pragma unroll
      for (int nt = 0; nt < NR; ++nt) {
        float *p = so + (warp * kRows + 8 * nt + 2 * tq) * L_::PAD + (D == 128 ? 16 : 8) * g + 2 * mt;
        if (rg * kRows + 8 * nt + 2 * tq >= a.QPK) continue;
        *reinterpret_cast<float2 *>(p) = make_float2(ot[mt][nt][0], ot[mt][nt][2]);
        *reinterpret_cast<float2 *>(p + L_::PAD) = make_float2(ot[mt][nt][1], ot[mt][nt][3]);
      }
  } else {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float *p = so + (warp * kRows + g) * L_::PAD + 8 * n + 2 * tq;
      if (valid[0]) *reinterpret_cast<float2 *>(p) = make_float2(o[n][0], o[n][1]);
      if constexpr (!HALF)
        if (valid[1])
          *reinterpret_cast<float2 *>(p + 8 * L_::PAD) = make_float2(o[n][2], o[n][3]);
    }
  }
  __syncthreads();
  const int rows = min(a.QPK - rg * kRows, kRows);
  uint16_t *out = static_cast<uint16_t *>(a.out) +
                  (static_cast<int64_t>(b) * a.H + kvh * a.QPK + rg * kRows) * D;
  for (int i = threadIdx.x; i < rows * D; i += kThreads) {
    const int r = i / D, d = i % D;
    float M = -INFINITY, num = 0.f, den = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm[w * kRows + r]);
    if (M != -INFINITY) {
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float e = fast_exp2(sm[w * kRows + r] - M);
        num = fmaf(e, so[(w * kRows + r) * L_::PAD + d], num);
        den = fmaf(e, sl[w * kRows + r], den);
      }
    }
    if (a.parts == 1) {
      const float v = joined(M, num, den) * a.v_scale;
      out[i] = static_cast<uint16_t>(T::from_f2(v, 0.f) & 0xffffu);
    } else {
      so[(kWarps * kRows + r) * L_::PAD + d] = num;
      if (d == 0) {
        sm[kWarps * kRows + r] = M;
        sl[kWarps * kRows + r] = den;
      }
    }
  }
  if (a.parts == 1) return;
  cluster_sync();
  for (int i = part * kThreads + threadIdx.x; i < rows * D; i += a.parts * kThreads) {
    const int r = i / D, d = i % D;
    float pm[kMaxParts], pl[kMaxParts], po[kMaxParts], M = -INFINITY, num = 0.f, den = 0.f;
#pragma unroll
    for (int c = 0; c < kMaxParts; ++c) {
      const uint32_t from = min(c, a.parts - 1);
      pm[c] = cluster_loadf(sm + kWarps * kRows + r, from);
      pl[c] = cluster_loadf(sl + kWarps * kRows + r, from);
      po[c] = cluster_loadf(so + (kWarps * kRows + r) * L_::PAD + d, from);
    }
#pragma unroll
    for (int c = 0; c < kMaxParts; ++c) M = fmaxf(M, pm[c]);
    if (M != -INFINITY) {
#pragma unroll
      for (int c = 0; c < kMaxParts; ++c) {
        if (c >= a.parts) break;
        const float e = fast_exp2(pm[c] - M);
        num = fmaf(e, po[c], num);
        den = fmaf(e, pl[c], den);
      }
    }
    const float v = joined(M, num, den) * a.v_scale;
    out[i] = static_cast<uint16_t>(T::from_f2(v, 0.f) & 0xffffu);
  }
  cluster_sync();  // no CTA leaves while its shared memory is read
}

template <class T, int D, bool KV8, int ROWS, int W>
static cudaError_t launch_w(const Args &a, const CUtensorMap &tmap, int num_seqs,
                            cudaStream_t stream) {
  auto kern = sparse_kernel<T, D, KV8, ROWS, W>;
  constexpr int smem = Lay<D, KV8, W>::SMEM;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_shared_memory(kern, allowed, 1024);
  if (e != cudaSuccess) return e;
  PdlLaunch cfg(dim3(a.parts, a.KVH * a.row_groups, num_seqs), 32 * W, smem, stream, a.parts);
  return cudaLaunchKernelEx(&cfg.c, kern, a, tmap);
}

template <class T, int D, bool KV8, int W>
static cudaError_t launch_rows(const Args &a, const CUtensorMap &tmap, int num_seqs,
                               cudaStream_t stream) {
  if constexpr (KV8)
    if (a.QPK <= 4) return launch_w<T, D, KV8, 4, W>(a, tmap, num_seqs, stream);
  return a.QPK <= 8 ? launch_w<T, D, KV8, 8, W>(a, tmap, num_seqs, stream)
                    : launch_w<T, D, KV8, 16, W>(a, tmap, num_seqs, stream);
}

template <class T, int D, bool KV8>
static cudaError_t launch_typed(const Args &a, const CUtensorMap &tmap, int num_seqs, bool few,
                                cudaStream_t stream) {
  return few ? launch_rows<T, D, KV8, kFew>(a, tmap, num_seqs, stream)
             : launch_rows<T, D, KV8, kMany<D, KV8>>(a, tmap, num_seqs, stream);
}

}  // namespace sparse

cudaError_t launch_sparse_decode(void *out, const void *query, int num_seqs, const void *kv_cache,
                                 const int32_t *block_tables, int max_blocks_per_seq,
                                 const int32_t *seq_lens, const int32_t *selected,
                                 int max_selected, const Geometry &g, cudaStream_t stream) {
  DeviceInfo dev;
  cudaError_t e = current_device_info(&dev);
  if (e != cudaSuccess) return e;
  CUtensorMap tmap;
  const cuuint64_t eb = static_cast<cuuint64_t>(g.elem_bytes);
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(g.D), static_cast<cuuint64_t>(g.KVH),
                              static_cast<cuuint64_t>(g.num_blocks * g.BS), 2};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(g.D) * eb,
                                 static_cast<cuuint64_t>(g.row_bytes),
                                 static_cast<cuuint64_t>(g.num_blocks * g.block_bytes)};
  const cuuint32_t box[4] = {g.fp8 ? static_cast<cuuint32_t>(g.D) : 64u, 1,
                             static_cast<cuuint32_t>(sparse::kUnit), 1};
  const bool bf = g.dtype == PKV_BF16;
  const CUtensorMapDataType dt =
      g.fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
            : (bf ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16);
  const CUtensorMapSwizzle swz =
      !g.fp8 || g.D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  // no wider fetches than a head's row: the next head's rows of this block are
  // read only if it selected the block too
  const cuuint64_t row = static_cast<cuuint64_t>(g.D) * eb;
  const CUtensorMapL2promotion promotion =
      row >= 256   ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
      : row == 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
                   : CU_TENSOR_MAP_L2_PROMOTION_L2_64B;
  if (encode_tensor_map(&tmap, dt, 4, const_cast<void *>(kv_cache), dims, strides, box, swz,
                        promotion) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  sparse::Args a{};
  a.out = out;
  a.query = static_cast<const uint16_t *>(query);
  a.block_tables = block_tables;
  a.seq_lens = seq_lens;
  a.selected = selected;
  a.alibi = g.alibi;
  a.num_blocks = g.num_blocks;
  a.max_blocks_per_seq = max_blocks_per_seq;
  a.max_selected = max_selected;
  a.H = g.H;
  a.KVH = g.KVH;
  a.QPK = g.QPK;
  a.BS = g.BS;
  a.window = g.window;
  a.row_groups = (g.QPK + sparse::kRows - 1) / sparse::kRows;
  a.scale_log2 = g.scale * kLog2e * g.k_scale;
  a.v_scale = g.v_scale;
  const int64_t items = static_cast<int64_t>(num_seqs) * g.KVH * a.row_groups;
  const int64_t units =
      static_cast<int64_t>(std::min(max_selected, max_blocks_per_seq)) * (g.BS / sparse::kUnit);
  // Measured (2048 keys of 8 or 16 KV heads, us): 8-warp CTAs, one to an SM, are
  // faster up to a CTA per SM (128 items: 26 / 28 and 16 / 17 against the best of
  // the others), with as many parts as then fit (8 items: 14 / 10 / 8 / 7 in 1 / 2 /
  // 4 / 8 parts); clusters of 8 such CTAs fit a GPC's SMs badly (16 of them: 13
  // against 8 in fours).  From there on parts only add prologues and joins (512
  // items: 90 / 91 / 101 / 116), but for 8-bit caches at half a wave (256 items:
  // 36 / 32, 16-bit 49 / 50).
  const bool few = items <= dev.sms;
  if (few) {
    a.parts = items * 8 <= dev.sms / 2 ? 8 : items * 4 <= dev.sms ? 4 : items * 2 <= dev.sms ? 2 : 1;
    while (a.parts > 1 && units < a.parts * sparse::kFew) a.parts /= 2;
  } else {
    a.parts = items * 2 <= 4LL * dev.sms ? 2 : 1;
  }
#define PKV_SP(TT, DD)                                                                \
  if (g.D == DD)                                                                      \
    return g.fp8 ? sparse::launch_typed<TT, DD, true>(a, tmap, num_seqs, few, stream)      \
                 : sparse::launch_typed<TT, DD, false>(a, tmap, num_seqs, few, stream);
  if (bf) {
    PKV_SP(BF16, 128) PKV_SP(BF16, 64)
  } else {
    PKV_SP(FP16, 128) PKV_SP(FP16, 64)
  }
#undef PKV_SP
  return cudaErrorInvalidValue;
}

cudaError_t read_device_error_sparse(unsigned long long *out) {
  return read_and_clear_unit_error(out);
}

}  // namespace pkv
