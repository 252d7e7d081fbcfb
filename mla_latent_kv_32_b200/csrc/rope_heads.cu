// mla_rope_heads: the rotation of `dim` values of every head of a token row,
//   y0 = x0 cos - x1 sin,  y1 = x1 cos + x0 sin,
// for the pairs (2j, 2j+1) (interleaved) or (j, j + dim/2) (half) with angle j
// of the token's table row ("Deconstructing DeepSeek V4 Pro ...", section
// "Hands-On PyTorch Implementation", apply_rope): float32, each product and
// sum rounded once, then bf16, as the cache's keys are turned.
//
// A thread owns 8 pairs (two 16-byte pieces of a head) of kHeads heads of one
// token: the 16 table values are read once for them, and all its loads are in
// flight together. Neighbouring threads own neighbouring pieces, then
// neighbouring heads, so a warp's accesses are contiguous where the rows are.
// Bound: HBM for many tokens (4099 x 128 heads of 64: 23.0 us, 5.9 TB/s, an
// elementwise pass over as many bytes takes 21.7), the launch for few (64 x 128 heads:
// 2.2 us).
#include "internal.h"
#include "sm100.cuh"

namespace mla {
namespace {

using sm100::cvt_bf16x2;

constexpr int kThreads = 128;
// heads per thread: 1, 2, 4 take 27.0, 24.1, 22.5 us on 4099 x 128 heads in one sweep,
// 26.5, 22.3, 23.0 in another
constexpr int kHeads = 4;

__device__ __forceinline__ void turn8(const uint4 &a, const uint4 &b, const float4 (&cs)[4],
                                      bool half, uint4 &oa, uint4 &ob) {
  const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
  const float cosv[8] = {cs[0].x, cs[0].z, cs[1].x, cs[1].z, cs[2].x, cs[2].z, cs[3].x, cs[3].z};
  const float sinv[8] = {cs[0].y, cs[0].w, cs[1].y, cs[1].w, cs[2].y, cs[2].w, cs[3].y, cs[3].w};
  uint32_t ra[4], rb[4];
  if (half) {
    // a = the 8 first values of the pairs, b = the 8 second ones
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float y0, y1, z0, z1;
      rope_pair_rn(bf16_bits_to_f32(wa[i] & 0xFFFFu), bf16_bits_to_f32(wb[i] & 0xFFFFu),
                   cosv[2 * i], sinv[2 * i], y0, y1);
      rope_pair_rn(bf16_bits_to_f32(wa[i] >> 16), bf16_bits_to_f32(wb[i] >> 16), cosv[2 * i + 1],
                   sinv[2 * i + 1], z0, z1);
      ra[i] = cvt_bf16x2(y0, z0);
      rb[i] = cvt_bf16x2(y1, z1);
    }
  } else {
    // a = pairs 0..3, b = pairs 4..7
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float y0, y1;
      rope_pair_rn(bf16_bits_to_f32(wa[i] & 0xFFFFu), bf16_bits_to_f32(wa[i] >> 16), cosv[i],
                   sinv[i], y0, y1);
      ra[i] = cvt_bf16x2(y0, y1);
      rope_pair_rn(bf16_bits_to_f32(wb[i] & 0xFFFFu), bf16_bits_to_f32(wb[i] >> 16), cosv[4 + i],
                   sinv[4 + i], y0, y1);
      rb[i] = cvt_bf16x2(y0, y1);
    }
  }
  oa = make_uint4(ra[0], ra[1], ra[2], ra[3]);
  ob = make_uint4(rb[0], rb[1], rb[2], rb[3]);
}

// x may be out itself (the same rows): a thread reads its pieces before it
// writes them and no other thread touches them, so no load is through the
// read-only path.
__global__ void __launch_bounds__(kThreads) rope_heads_kernel(const RopeHeadsArgs a) {
  const int pieces = a.dim >> 4;
  const int groups = (a.n_h + kHeads - 1) / kHeads;
  const long long unit = (long long)blockIdx.x * kThreads + threadIdx.x;
  const long long per_token = (long long)groups * pieces;
  if (unit >= (long long)a.T * per_token) return;
  const int t = (int)(unit / per_token);
  const int rest = (int)(unit - t * per_token);
  const int g = rest / pieces, piece = rest - g * pieces;
  const int p = __ldg(a.pos + t);
  // offsets of the unit's two 8-value pieces within a head
  const int o0 = a.half ? 8 * piece : 16 * piece;
  const int o1 = a.half ? (a.dim >> 1) + 8 * piece : 16 * piece + 8;
  const uint16_t *x = a.x + (long long)t * a.ld_x;
  uint4 u[kHeads], v[kHeads];
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    const int h = g + i * groups;
    if (h >= a.n_h) continue;
    const uint16_t *xh = x + (long long)h * a.hs_x;
    u[i] = *reinterpret_cast<const uint4 *>(xh + o0);
    v[i] = *reinterpret_cast<const uint4 *>(xh + o1);
  }
  if (p < 0 || p >= a.max_pos) {
    if (rest == 0) report(a.status, MLA_DEV_BAD_POSITION);
    return;
  }
  float4 cs[4];
  const float4 *row = reinterpret_cast<const float4 *>(a.rope_table + (size_t)p * a.dim) + 4 * piece;
#pragma unroll
  for (int i = 0; i < 4; ++i) cs[i] = __ldg(row + i);
  uint16_t *out = a.out + (long long)t * a.ld_o;
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    const int h = g + i * groups;
    if (h >= a.n_h) continue;
    uint4 y0, y1;
    turn8(u[i], v[i], cs, a.half != 0, y0, y1);
    uint16_t *oh = out + (long long)h * a.hs_o;
    *reinterpret_cast<uint4 *>(oh + o0) = y0;
    *reinterpret_cast<uint4 *>(oh + o1) = y1;
  }
}

}  // namespace

mla_status_t launch_rope_heads(const RopeHeadsArgs &a, cudaStream_t stream) {
  const long long units = (long long)a.T * ((a.n_h + kHeads - 1) / kHeads) * (a.dim >> 4);
  const long long blocks = (units + kThreads - 1) / kThreads;
  if (blocks > 0x7FFFFFFFll) return fail(MLA_ERR_UNSUPPORTED, "too many values to rotate");
  rope_heads_kernel<<<(unsigned)blocks, kThreads, 0, stream>>>(a);
  MLA_LAUNCH_CHECK("rope_heads_kernel");
  return MLA_OK;
}

}  // namespace mla
