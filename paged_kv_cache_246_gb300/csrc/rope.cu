// kv_cache_write_rope, kv_cache_write_rope_axes: the cache write with the rotary
// position embedding on the way.  Per pair (x1, x2) of channels and the position's cos c, sin s:
//     y1 = x1 c - x2 s,   y2 = x2 c + x1 s      (fp32, one rounding out)
// Queries go to query_out, keys (rotated) and values to their cache slots.
//
// Bound by HBM: a token's row is read once and written once (24 KB at 32 + 8
// + 8 heads of 128 and 16 bits), the rotation is 6 flops per pair.  A head is
// D / 16 lanes wide: a lane owns two 16-byte chunks whose channels pair up
// (half split: chunks i and i + rot_dim / 16; interleaved: any two), so no
// pair crosses lanes and every access is an aligned 16 bytes.
#include <cuda_fp8.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace pkv {
namespace rope {

struct Args {
  uint16_t *q_out;
  const uint16_t *q, *k, *v;
  int64_t q_out_stride, q_stride, k_stride, v_stride;  // elements
  int64_t num_tokens, max_position, num_slots;
  const int64_t *positions, *slots;
  const float *cos_sin;
  uint8_t *k_half, *v_half;
  int64_t row_bytes;  // of the cache
  int H, KVH, rot;
  float k_scale, v_scale, k_inv, v_inv;  // and their reciprocals (0: divide)
};

// Positions of several axes: elements from one axis to the next, and the axis
// of each of up to 64 pairs, 2 bits apiece.
struct Axes {
  int64_t stride;
  uint32_t bits[4];
};

__device__ __forceinline__ void widen(float (&f)[8], const uint4 &u, BF16) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = BF16::to_f2(w[i]);
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
  }
}
__device__ __forceinline__ void widen(float (&f)[8], const uint4 &u, FP16) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = FP16::to_f2(w[i]);
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
  }
}

template <class T>
__device__ __forceinline__ uint4 narrow(const float (&f)[8]) {
  return make_uint4(T::from_f2(f[0], f[1]), T::from_f2(f[2], f[3]), T::from_f2(f[4], f[5]),
                    T::from_f2(f[6], f[7]));
}

// x / scale as IEEE division rounds it, for inv = 1 / scale rounded and a scale in
// 2^-100 .. 2^100: the remainder of the first product corrects it (Markstein 1990).
// Quotients of 512 and more saturate as they are, zeros keep their sign (0x44000000
// is 512).
__device__ __forceinline__ float quotient(float x, float scale, float inv) {
  const float q = x * inv;
  const bool ordinary = __float_as_uint(fabsf(q)) - 1u < 0x44000000u - 1u;
  return ordinary ? fmaf(fmaf(-q, scale, x), inv, q) : q;
}

// Eight values as E4M3 codes of f / scale (fp32 quotient, nearest even,
// saturating), as the plain cache write makes them.
__device__ __forceinline__ uint2 codes8(const float (&f)[8], float scale, float inv) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // inv = 0: a scale outside that range
    const float2 q = inv != 0.f ? make_float2(quotient(f[2 * i], scale, inv),
                                              quotient(f[2 * i + 1], scale, inv))
                                : make_float2(__fdiv_rn(f[2 * i], scale),
                                              __fdiv_rn(f[2 * i + 1], scale));
    w[i] = __nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3);
  }
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// (x1, x2) -> (x1 c - x2 s, x2 c + x1 s)
__device__ __forceinline__ void rotate(float &x1, float &x2, float c, float s) {
  const float y1 = x1 * c - x2 * s, y2 = x2 * c + x1 * s;
  x1 = y1;
  x2 = y2;
}

// Item i of a token: two 16-byte chunks, c0 and c1, of one of its H + 2 KVH
// heads, and which of the two turn.
template <int D, bool INTER>
struct Item {
  static constexpr int LPH = D / 16;  // lanes per head
  int j, c0, c1, hh;
  bool rot0, rot1, is_q, is_v;
  __device__ __forceinline__ Item(const Args &a, int i) {
    const int head = i / LPH;
    j = i % LPH;
    if constexpr (INTER) {
      c0 = 2 * j;
      c1 = c0 + 1;
      rot0 = c0 * 8 < a.rot;
      rot1 = c1 * 8 < a.rot;
    } else {
      const int half = a.rot / 16;
      rot0 = rot1 = j < half;
      c0 = rot0 ? j : 2 * j;
      c1 = rot0 ? j + half : 2 * j + 1;
    }
    is_q = head < a.H;
    is_v = head >= a.H + a.KVH;
    hh = is_q ? head : is_v ? head - a.H - a.KVH : head - a.H;
  }
  template <bool BULK>
  __device__ __forceinline__ void load(const Args &a, int64_t t, uint4 &u0, uint4 &u1) const {
    const int64_t stride = is_q ? a.q_stride : is_v ? a.v_stride : a.k_stride;
    const uint4 *s4 =
        reinterpret_cast<const uint4 *>((is_q ? a.q : is_v ? a.v : a.k) + t * stride + hh * D);
    u0 = BULK ? __ldcs(s4 + c0) : s4[c0];
    u1 = BULK ? __ldcs(s4 + c1) : s4[c1];
  }
};

// Four cosines or sines of a row in global or in shared memory.
template <bool SHARED>
__device__ __forceinline__ float4 row4(const float *p) {
  return SHARED ? *reinterpret_cast<const float4 *>(p) : __ldg(reinterpret_cast<const float4 *>(p));
}

// The item's chunks turned by the row `cs` (rot / 2 cosines, then sines), and stored.
template <class T, int D, bool KV8, bool INTER, bool BULK, bool SHARED>
__device__ __forceinline__ void finish(const Args &a, const Item<D, INTER> &it, int64_t t,
                                       int64_t slot, const float *cs, uint4 u0, uint4 u1) {
  const int c0 = it.c0, c1 = it.c1;
  const bool turn = !it.is_v && (it.rot0 || it.rot1);
  if (turn || (KV8 && !it.is_q)) {
    float x0[8], x1[8];
    widen(x0, u0, T{});
    widen(x1, u1, T{});
    if (turn) {
      const int half = a.rot / 2;
      if constexpr (INTER) {
        // chunk c holds pairs 4c .. 4c + 3
        const float4 ca = row4<SHARED>(cs + 4 * c0), sa = row4<SHARED>(cs + half + 4 * c0);
        rotate(x0[0], x0[1], ca.x, sa.x);
        rotate(x0[2], x0[3], ca.y, sa.y);
        rotate(x0[4], x0[5], ca.z, sa.z);
        rotate(x0[6], x0[7], ca.w, sa.w);
        if (it.rot1) {
          const float4 cb = row4<SHARED>(cs + 4 * c1), sb = row4<SHARED>(cs + half + 4 * c1);
          rotate(x1[0], x1[1], cb.x, sb.x);
          rotate(x1[2], x1[3], cb.y, sb.y);
          rotate(x1[4], x1[5], cb.z, sb.z);
          rotate(x1[6], x1[7], cb.w, sb.w);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
          const float4 cc = row4<SHARED>(cs + 8 * it.j + e);
          const float4 ss = row4<SHARED>(cs + half + 8 * it.j + e);
          rotate(x0[e], x1[e], cc.x, ss.x);
          rotate(x0[e + 1], x1[e + 1], cc.y, ss.y);
          rotate(x0[e + 2], x1[e + 2], cc.z, ss.z);
          rotate(x0[e + 3], x1[e + 3], cc.w, ss.w);
        }
      }
    }
    if (KV8 && !it.is_q) {
      const float scale = it.is_v ? a.v_scale : a.k_scale;
      uint2 *d2 = reinterpret_cast<uint2 *>((it.is_v ? a.v_half : a.k_half) + slot * a.row_bytes +
                                            it.hh * D);
      const float inv = it.is_v ? a.v_inv : a.k_inv;
      const uint2 w0 = codes8(x0, scale, inv), w1 = codes8(x1, scale, inv);
      if constexpr (BULK) {
        __stcs(d2 + c0, w0);
        __stcs(d2 + c1, w1);
      } else {
        d2[c0] = w0;
        d2[c1] = w1;
      }
      return;
    }
    if (it.rot0) u0 = narrow<T>(x0);
    if (it.rot1) u1 = narrow<T>(x1);
  }
  uint4 *d4 = it.is_q ? reinterpret_cast<uint4 *>(a.q_out + t * a.q_out_stride + it.hh * D)
                      : reinterpret_cast<uint4 *>((it.is_v ? a.v_half : a.k_half) +
                                                  slot * a.row_bytes + it.hh * D * 2);
  if constexpr (BULK) {
    __stcs(d4 + c0, u0);
    __stcs(d4 + c1, u1);
  } else {
    d4[c0] = u0;
    d4[c1] = u1;
  }
}

// CTA = one token; thread i takes the lane slots i, i + blockDim, ... of the
// token's (H + 2 KVH) heads.  The row is loaded before slot and position are
// looked at (that of a token to be skipped is only read), so one memory latency
// covers all three.  Two or four tokens per CTA (81, 114 us for 16384 tokens of
// 48 heads of 128, against 74 with one) only cost resident threads.
//
// BULK, for more than 6 tokens per SM: CTAs of 192 threads and streaming loads
// and stores (the rows are more than L2 keeps).  Measured against 512 threads
// and plain accesses: 9.2 / 12.0 us for 2048 tokens, 31.8 / 40.2 for 8192, 61 /
// 78 for 16384 (6.7 TB/s); for 512 tokens 3.2 / 3.0 and for 64 2.3 / 1.9.  Registers
// for 8 such CTAs per SM: over an 8-bit cache 67 us for 16384 tokens, 71 with 5 or 6.
template <class T, int D, bool KV8, bool INTER, bool BULK>
__global__ void __launch_bounds__(BULK ? 192 : 512, BULK ? 8 : 1)
rope_write_kernel(const Args a) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t t = blockIdx.x;
  const int items = (a.H + 2 * a.KVH) * (D / 16);
  for (int i = threadIdx.x; i < items; i += blockDim.x) {
    const Item<D, INTER> it(a, i);
    uint4 u0, u1;
    it.template load<BULK>(a, t, u0, u1);
    const int64_t slot = __ldg(a.slots + t), pos = __ldg(a.positions + t);
    if (slot < 0) return;  // padding token
    if (slot >= a.num_slots || pos < 0 || pos >= a.max_position) {
      if (i == 0) record_error(PKV_ERR_BOUNDS, t);
      return;
    }
    finish<T, D, KV8, INTER, BULK, false>(a, it, t, slot, a.cos_sin + pos * a.rot, u0, u1);
  }
}

// Positions of several axes: the CTA first gathers its token's cosines and
// sines, each from its pair's own row of the table, into shared memory (the
// first items' rows are on their way meanwhile); from there the heads' lanes
// read them as the kernel above reads a table row.  The pairs' axes, 2 bits
// each, are launch arguments.
//
// BULK: CTAs of 96 threads, 16 to an SM: while one waits for its table rows
// others move theirs.  16384 tokens of 48 heads of 128: 65 us (6.3 TB/s), with
// 192 threads 71, with 64 65, with 384 80; into an 8-bit cache 64 / 68 / 64 / 83.
// Two of a thread's items loaded ahead spill (105), a row gathered by each warp
// instead of the barrier is equal (71 against 71).
template <class T, int D, bool KV8, bool INTER, bool BULK>
__global__ void __launch_bounds__(BULK ? 96 : 512, BULK ? 16 : 1)
rope_axes_write_kernel(const Args a, const Axes x) {
  __shared__ __align__(16) float row[128];
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t t = blockIdx.x;
  const int items = (a.H + 2 * a.KVH) * (D / 16);
  int i = threadIdx.x;
  uint4 u0 = make_uint4(0, 0, 0, 0), u1 = u0;
  if (i < items) Item<D, INTER>(a, i).template load<BULK>(a, t, u0, u1);
  const int64_t slot = __ldg(a.slots + t);
  bool bad = slot >= a.num_slots;
  const int half = a.rot / 2;
  for (int p = threadIdx.x; p < a.rot; p += blockDim.x) {
    const int pair = p < half ? p : p - half;
    const uint32_t axis = (x.bits[pair / 16] >> (2 * (pair % 16))) & 3u;
    const int64_t pos = __ldg(a.positions + axis * x.stride + t);
    if (pos < 0 || pos >= a.max_position)
      bad = true;
    else
      row[p] = __ldg(a.cos_sin + pos * a.rot + p);
  }
  bad = __syncthreads_or(bad);
  if (slot < 0) return;  // padding token
  if (bad) {
    if (threadIdx.x == 0) record_error(PKV_ERR_BOUNDS, t);
    return;
  }
  while (i < items) {
    finish<T, D, KV8, INTER, BULK, true>(a, Item<D, INTER>(a, i), t, slot, row, u0, u1);
    i += blockDim.x;
    if (i < items) Item<D, INTER>(a, i).template load<BULK>(a, t, u0, u1);
  }
}

template <class T, int D, bool KV8>
static cudaError_t launch_typed(const Args &a, const Axes *x, bool interleaved,
                                cudaStream_t stream) {
  const int items = (a.H + 2 * a.KVH) * (D / 16);
  DeviceInfo dev;
  cudaError_t e = current_device_info(&dev);
  if (e != cudaSuccess) return e;
  const bool bulk = a.num_tokens > 6LL * dev.sms;
  PdlLaunch cfg(dim3(static_cast<unsigned>(a.num_tokens)),
                std::min(!bulk ? 512 : x ? 96 : 192, (items + 31) / 32 * 32), 0, stream);
#define PKV_ROPE_FORM(IN, BULK)                                                             \
  return x ? cudaLaunchKernelEx(&cfg.c, rope_axes_write_kernel<T, D, KV8, IN, BULK>, a, *x) \
           : cudaLaunchKernelEx(&cfg.c, rope_write_kernel<T, D, KV8, IN, BULK>, a)
  if (bulk && interleaved) PKV_ROPE_FORM(true, true);
  if (bulk) PKV_ROPE_FORM(false, true);
  if (interleaved) PKV_ROPE_FORM(true, false);
  PKV_ROPE_FORM(false, false);
#undef PKV_ROPE_FORM
}

}  // namespace rope

cudaError_t launch_rope_write(const RopeCall &r, const Geometry &g, cudaStream_t stream) {
  rope::Args a{};
  a.q_out = static_cast<uint16_t *>(r.query_out);
  a.q = static_cast<const uint16_t *>(r.query);
  a.k = static_cast<const uint16_t *>(r.key);
  a.v = static_cast<const uint16_t *>(r.value);
  a.q_out_stride = r.query_out_stride;
  a.q_stride = r.query_stride;
  a.k_stride = r.key_stride;
  a.v_stride = r.value_stride;
  a.num_tokens = r.num_tokens;
  a.max_position = r.max_position;
  a.num_slots = g.num_blocks * g.BS;
  a.positions = r.positions;
  a.slots = r.slot_mapping;
  a.cos_sin = r.cos_sin;
  a.k_half = static_cast<uint8_t *>(r.kv_cache);
  a.v_half = a.k_half + g.num_blocks * g.block_bytes;
  a.row_bytes = g.row_bytes;
  a.H = g.H;
  a.KVH = g.KVH;
  a.rot = r.rot_dim;
  a.k_scale = g.k_scale;
  a.v_scale = g.v_scale;
  auto inverse = [](float x) { return x >= 0x1p-100f && x <= 0x1p100f ? 1.f / x : 0.f; };
  a.k_inv = inverse(g.k_scale);
  a.v_inv = inverse(g.v_scale);
  rope::Axes x = {r.positions_stride, {0, 0, 0, 0}};
  if (r.pair_axes)
    for (int i = 0; i < r.rot_dim / 2; ++i)
      x.bits[i / 16] |= static_cast<uint32_t>(r.pair_axes[i]) << (2 * (i % 16));
  const rope::Axes *axes = r.pair_axes ? &x : nullptr;
  const bool bf = g.dtype == PKV_BF16, in = r.interleaved != 0;
#define PKV_ROPE(TT, DD)                                                     \
  if (g.D == DD)                                                             \
    return g.fp8 ? rope::launch_typed<TT, DD, true>(a, axes, in, stream)     \
                 : rope::launch_typed<TT, DD, false>(a, axes, in, stream);
  if (bf) {
    PKV_ROPE(BF16, 128) PKV_ROPE(BF16, 64)
  } else {
    PKV_ROPE(FP16, 128) PKV_ROPE(FP16, 64)
  }
#undef PKV_ROPE
  return cudaErrorInvalidValue;
}

cudaError_t read_device_error_rope(unsigned long long *out) { return read_and_clear_unit_error(out); }

}  // namespace pkv
