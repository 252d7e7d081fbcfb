// mla_norm_append[_fp8]: what stands between a layer's down-projections and
// its cache, in one pass over the tokens:
//   c  = c^KV / sqrt(mean(c^KV^2) + eps) * w_kv      (512 wide) -> the cache
//   k  = RoPE(k^R, pos)                                         -> the cache
//   q  = c^Q  / sqrt(mean(c^Q^2)  + eps) * w_q       (q_dim wide, optional)
//
// One warp per token and side: a row's values stay in the warp's registers
// between the sum of squares and the scaling, so each is read once. The query
// side (when there is one) is the neighbouring warp, so that the two halves of
// a fused down-projection's row are read together. A lane issues all 16-byte
// loads of its row before it uses the first. Bound: HBM for many tokens (16381
// with q_dim 1536, 142.6 MB: 25.6 us, 5.6 TB/s), the launch and three dependent
// memory round trips (position, page id, store) for few (64: 1.9 us).
// Sums of squares, the mean and the scaled values are float32; each output is
// rounded once (bf16 nearest even, or E4M3 of the float32 value).
#include "internal.h"
#include "sm100.cuh"

namespace mla {
namespace {

using sm100::cvt_bf16x2;

constexpr int kWarpsPerCta = 4;
constexpr int kCtasPerSm = 10;   // 48 registers a thread, no spills

__device__ __forceinline__ void unpack8(const uint4 &v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16_bits_to_f32(w[i] & 0xFFFFu);
    x[2 * i + 1] = bf16_bits_to_f32(w[i] >> 16);
  }
}

__device__ __forceinline__ float square_sum8(const uint4 &v) {
  float x[8];
  unpack8(v, x);
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s = fmaf(x[i], x[i], s);
  return s;
}

// y = x * r * w for 8 values
__device__ __forceinline__ void scaled8(const uint4 &v, float r, const uint4 &w, float (&y)[8]) {
  float wv[8];
  unpack8(v, y);
  unpack8(w, wv);
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = y[i] * r * wv[i];
}

// 8 weights; w == nullptr: all ones
__device__ __forceinline__ uint4 load_weights(const uint16_t *w, int at) {
  return w != nullptr ? __ldg(reinterpret_cast<const uint4 *>(w + at))
                      : make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
}

__device__ __forceinline__ uint4 pack8(const float (&y)[8]) {
  return make_uint4(cvt_bf16x2(y[0], y[1]), cvt_bf16x2(y[2], y[3]), cvt_bf16x2(y[4], y[5]),
                    cvt_bf16x2(y[6], y[7]));
}

// Few tokens (kEarly): the weights are read with the row, so that they do not add
// a round trip to the chain of loads. Many: they are read (from L1) when the norm
// is known, and the row is unpacked twice, since held from the start they and the
// unpacked floats would take two thirds of the resident warps.
template <bool kEarly>
__device__ __forceinline__ const uint16_t *known(const uint16_t *w, float r) {
  if (!kEarly) asm volatile("" : "+l"(w) : "f"(r));
  return w;
}
template <bool kEarly>
__device__ __forceinline__ void repacked(uint4 &v) {
  if (!kEarly) asm volatile("" : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// One warp norms one query latent. The first kHeld chunks of a lane (q_dim up
// to 1536) stay in registers; a longer row's remaining chunks are read again.
constexpr int kHeld = 6;

template <bool kEarly>
__device__ __forceinline__ void norm_query_warp(const NormAppendArgs &a, int t, int lane) {
  const uint16_t *src = a.c_q + (size_t)t * a.ld_q;
  uint16_t *dst = a.q_out + (size_t)t * a.ld_qo;
  const int chunks = a.q_dim >> 3;
  uint4 v[kHeld], w[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int c = lane + 32 * i;
    v[i] = c < chunks ? *reinterpret_cast<const uint4 *>(src + 8 * c) : make_uint4(0, 0, 0, 0);
    if (kEarly && c < chunks) w[i] = load_weights(a.w_q, 8 * c);
  }
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) s += square_sum8(v[i]);
  for (int c = lane + 32 * kHeld; c < chunks; c += 32)
    s += square_sum8(*reinterpret_cast<const uint4 *>(src + 8 * c));
  const float r = rsqrtf(warp_sum(s) / (float)a.q_dim + a.eps);
  const uint16_t *wq = known<kEarly>(a.w_q, r);
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int c = lane + 32 * i;
    if (c >= chunks) continue;
    float y[8];
    repacked<kEarly>(v[i]);
    scaled8(v[i], r, kEarly ? w[i] : load_weights(wq, 8 * c), y);
    *reinterpret_cast<uint4 *>(dst + 8 * c) = pack8(y);
  }
  for (int c = lane + 32 * kHeld; c < chunks; c += 32) {
    float y[8];
    scaled8(*reinterpret_cast<const uint4 *>(src + 8 * c), r, load_weights(wq, 8 * c), y);
    *reinterpret_cast<uint4 *>(dst + 8 * c) = pack8(y);
  }
}

// Lanes 0..7 turn k^R, lane l the pairs [4 l, 4 l + 4): neighbours (2j, 2j+1)
// in 16 bytes, or, in the half layout, (j, j + 32) in two 8-byte halves. The
// arithmetic is the bf16 cache's (float32, each product and sum rounded once).
__device__ __forceinline__ void turn_key(const NormAppendArgs &a, const uint4 &kv, const float4 &cs0,
                                         const float4 &cs1, int lane, uint16_t *dst) {
  const float cosv[4] = {cs0.x, cs0.z, cs1.x, cs1.z};
  const float sinv[4] = {cs0.y, cs0.w, cs1.y, cs1.w};
  float x[8];
  unpack8(kv, x);
  float y[8];
  if (a.half) {
    // x[0..3] = values 4 l .. 4 l + 3, x[4..7] = values 32 + 4 l ..
#pragma unroll
    for (int i = 0; i < 4; ++i) rope_pair_rn(x[i], x[4 + i], cosv[i], sinv[i], y[i], y[4 + i]);
    *reinterpret_cast<uint2 *>(dst + 4 * lane) =
        make_uint2(cvt_bf16x2(y[0], y[1]), cvt_bf16x2(y[2], y[3]));
    *reinterpret_cast<uint2 *>(dst + MLA_D_R / 2 + 4 * lane) =
        make_uint2(cvt_bf16x2(y[4], y[5]), cvt_bf16x2(y[6], y[7]));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      rope_pair_rn(x[2 * i], x[2 * i + 1], cosv[i], sinv[i], y[2 * i], y[2 * i + 1]);
    *reinterpret_cast<uint4 *>(dst + 8 * lane) = pack8(y);
  }
}

template <bool kFp8, bool kEarly>
__global__ void __launch_bounds__(kWarpsPerCta * 32, kEarly ? 1 : kCtasPerSm)
norm_append_kernel(const NormAppendArgs a) {
  const long long w = (long long)blockIdx.x * kWarpsPerCta + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int t = (int)(a.q_dim > 0 ? w >> 1 : w);
  if (t >= a.n_tokens) return;
  if (a.q_dim > 0 && (w & 1)) {
    norm_query_warp<kEarly>(a, t, lane);
    return;
  }
  const int b = __ldg(a.seq_idx + t);
  const int p = __ldg(a.pos + t);
  // the row's values do not wait for the position
  const uint16_t *src = a.c_kv + (size_t)t * a.ld_c;
  // A lane's two chunks of 8 values: 16 codes of the FP8 row are one store, bf16 rows
  // go in two contiguous stores of the warp (with pairs of chunks a lane 10.0 us instead
  // of 9.5 for 16381 tokens without the query side).
  const int c0 = kFp8 ? 2 * lane : lane, c1 = kFp8 ? 2 * lane + 1 : 32 + lane;
  uint4 v0 = __ldg(reinterpret_cast<const uint4 *>(src) + c0);
  uint4 v1 = __ldg(reinterpret_cast<const uint4 *>(src) + c1);
  uint4 w0, w1;
  if (kEarly) {
    w0 = load_weights(a.w_kv, 8 * c0);
    w1 = load_weights(a.w_kv, 8 * c1);
  }
  uint4 kv = make_uint4(0, 0, 0, 0);
  if (lane < 8) {
    const uint16_t *k = a.k_pe + (size_t)t * a.ld_k;
    if (a.half) {
      const uint2 lo = __ldg(reinterpret_cast<const uint2 *>(k + 4 * lane));
      const uint2 hi = __ldg(reinterpret_cast<const uint2 *>(k + MLA_D_R / 2 + 4 * lane));
      kv = make_uint4(lo.x, lo.y, hi.x, hi.y);
    } else {
      kv = __ldg(reinterpret_cast<const uint4 *>(k) + lane);
    }
  }
  if (p < 0 || p >= a.max_pos || (p >> 6) >= a.max_pages) {
    if (lane == 0) report(a.status, MLA_DEV_BAD_POSITION);
    return;
  }
  if (b < 0 || b >= a.batch) {
    if (lane == 0) report(a.status, MLA_DEV_BAD_PAGE);
    return;
  }
  const int page = __ldg(a.block_table + (size_t)b * a.max_pages + (p >> 6));
  float4 cs0 = make_float4(0, 0, 0, 0), cs1 = cs0;
  if (lane < 8) {
    const float4 *row = reinterpret_cast<const float4 *>(a.rope_table + (size_t)p * MLA_D_R);
    cs0 = __ldg(row + 2 * lane);
    cs1 = __ldg(row + 2 * lane + 1);
  }
  if (page < 0 || page >= a.num_pages) {
    if (lane == 0) report(a.status, MLA_DEV_BAD_PAGE);
    return;
  }
  const float r = rsqrtf(warp_sum(square_sum8(v0) + square_sum8(v1)) / (float)MLA_D_C + a.eps);
  const uint16_t *wk = known<kEarly>(a.w_kv, r);
  if (!kEarly) {
    w0 = load_weights(wk, 8 * c0);
    w1 = load_weights(wk, 8 * c1);
  }
  float y[16];
  {
    float y0[8], y1[8];
    repacked<kEarly>(v0);
    repacked<kEarly>(v1);
    scaled8(v0, r, w0, y0);
    scaled8(v1, r, w1, y1);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y[i] = y0[i];
      y[8 + i] = y1[i];
    }
  }
  const size_t slot = (size_t)page * MLA_PAGE + (p & 63);
  if constexpr (kFp8) {
    // The scale and codes of the FP8 cache (the least 2^k with max / 2^k <=
    // 448, then E4M3 nearest even), taken of the float32 values: no bf16
    // rounding in between.
    uint8_t *dst = a.cache8 + slot * kFp8RowBytes;
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(y[i]));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
    int k = 0;
    if (amax > 0.f) {
      int e;
      const float m = frexpf(amax, &e);   // amax = m 2^e, m in [0.5, 1); 448 = 0.875 2^9
      k = m <= 0.875f ? e - 9 : e - 8;
    }
    // 2^-k as a float; two factors where it has none (k < -126)
    const int k1 = max(k, -126);
    const float f = __int_as_float((127 - k1) << 23);
    if (k1 != k) {
#pragma unroll
      for (int i = 0; i < 16; ++i) y[i] = ldexpf(y[i], k1 - k);
    }
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t lo, hi;
      const float a0 = y[4 * i] * f, a1 = y[4 * i + 1] * f;
      const float a2 = y[4 * i + 2] * f, a3 = y[4 * i + 3] * f;
      asm("{\n\t.reg .b16 r;\n\tcvt.rn.satfinite.e4m3x2.f32 r, %1, %2;\n\tcvt.u32.u16 %0, r;\n\t}"
          : "=r"(lo) : "f"(a1), "f"(a0));
      asm("{\n\t.reg .b16 r;\n\tcvt.rn.satfinite.e4m3x2.f32 r, %1, %2;\n\tcvt.u32.u16 %0, r;\n\t}"
          : "=r"(hi) : "f"(a3), "f"(a2));
      q[i] = lo | (hi << 16);
    }
    reinterpret_cast<uint4 *>(dst)[lane] = make_uint4(q[0], q[1], q[2], q[3]);
    if (lane == 0) a.scales8[slot] = ldexpf(1.f, k);
    if (lane < 8) turn_key(a, kv, cs0, cs1, lane, reinterpret_cast<uint16_t *>(dst + MLA_D_C));
  } else {
    uint16_t *dst = a.cache + slot * MLA_ROW;
    float y0[8], y1[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y0[i] = y[i];
      y1[i] = y[8 + i];
    }
    reinterpret_cast<uint4 *>(dst)[c0] = pack8(y0);
    reinterpret_cast<uint4 *>(dst)[c1] = pack8(y1);
    if (lane < 8) turn_key(a, kv, cs0, cs1, lane, dst + MLA_D_C);
  }
}

}  // namespace

mla_status_t launch_norm_append(const NormAppendArgs &a, cudaStream_t stream) {
  const long long warps = (long long)a.n_tokens * (a.q_dim > 0 ? 2 : 1);
  const unsigned grid = (unsigned)((warps + kWarpsPerCta - 1) / kWarpsPerCta);
  // One wave even with few resident warps: the shorter chain (64 tokens with
  // q_dim 1536: 1.9 against 3.1 us); else more warps (16381: 25.6 against 30.3).
  int sms = 0;
  mla_status_t st = device_info(&sms, nullptr, nullptr);
  if (st != MLA_OK) return st;
  const bool early = grid <= 4u * sms;
  auto kernel = a.cache8 != nullptr
                    ? (early ? norm_append_kernel<true, true> : norm_append_kernel<true, false>)
                    : (early ? norm_append_kernel<false, true> : norm_append_kernel<false, false>);
  kernel<<<grid, kWarpsPerCta * 32, 0, stream>>>(a);
  MLA_LAUNCH_CHECK("norm_append_kernel");
  return MLA_OK;
}

}  // namespace mla
