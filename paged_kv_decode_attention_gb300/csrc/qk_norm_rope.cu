// qk_norm_rope.cu -- what stands between a layer's QKV projection and its
// attention, in one pass: RMS norm of every query and key head, rotation by
// the token's position, and the append of K and V ("Chapter 8: Inference
// Optimization" (clxhxhhr.top/posts/4341), §8.1.1: a step stores the K and V
// of the token it processes; §8.3.1: slot = physical block x 16 + offset; the
// stored formats are those of §8.4.2 and §8.4.4).
//
// Mathematics, per head vector x of 128 values (FP32 throughout):
//   y   = x * rsqrt(mean(x^2) + eps) * w          (without a weight: y = x)
//   z_a = y_a cos - y_b sin,  z_b = y_b cos + y_a sin   for each rotated pair
// with (a, b) = (i, i + rot/2) or (2i, 2i + 1), and one rounding at the end:
// to BF16 (queries; BF16 pools), to E4M3 (nearest even, saturating) or to
// q8_0.  V is stored as the append stores it.
//
// What bounds it: HBM for many tokens (each value read once and written once;
// the FP32 work is about 10 instructions per value), launch latency for few.
// Layout: 16 lanes per (token, KV head), each 8 consecutive dims (one 16-byte
// access per row), taking the group's 4 query heads, its K and its V.  All
// six rows are loaded before the first is used, the cosines and sines of the
// lane's dims are read once for five rows, and a row's reductions and its
// exchange of the rotation partner stay inside the 16 lanes.  A CTA is one
// warp: nothing is shared between warps, and an SM's slots refill one by one
// (4 x 8192 tokens: 134.5 us = 6.1 TB/s; with 128 threads 141, with 256 162;
// a grid that stays and loads ahead 175: fewer warps fit).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "pkv_common.cuh"
#include "pkv_kernels.h"

namespace pkv {
namespace {

constexpr int kLanes = 16;                  // lanes per (token, KV head)
constexpr int kPerLane = kHeadDim / kLanes;  // 8 dims
constexpr int kRopeThreads = 32;  // two (token, KV head) items

__device__ __forceinline__ void unpack8(const uint4 v, float* f) {
  f[0] = bf16_lo(v.x);
  f[1] = bf16_hi(v.x);
  f[2] = bf16_lo(v.y);
  f[3] = bf16_hi(v.y);
  f[4] = bf16_lo(v.z);
  f[5] = bf16_hi(v.z);
  f[6] = bf16_lo(v.w);
  f[7] = bf16_hi(v.w);
}

__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

// Store one row's 8 values of this lane into slot (blk, off) of a pool.
template <int kFormat>
__device__ __forceinline__ void store_row(uint8_t* pool, int64_t tile, int off, int c, const float* f) {
  if constexpr (kFormat == PKV_KV_BF16) {
    reinterpret_cast<uint4*>(pool + tile * kTileBytes)[off * kLanes + c] = pack8(f);
  } else if constexpr (kFormat == PKV_KV_FP8_E4M3) {
    uint32_t pairs[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint16_t p2;
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(p2) : "f"(f[2 * e + 1]), "f"(f[2 * e]));
      pairs[e] = p2;
    }
    reinterpret_cast<uint2*>(pool + tile * kFp8TileBytes)[off * kLanes + c] =
        make_uint2(pairs[0] | (pairs[1] << 16), pairs[2] | (pairs[3] << 16));
  } else {
    // q8_0: the rule of q8_0_quantize_lane, 4 lanes x 8 values per group of 32
    float amax = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(f[e]));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const float d = __fdiv_rn(amax, 127.0f);
    const float id = d != 0.0f ? __fdiv_rn(1.0f, d) : 0.0f;
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int code = static_cast<int>(roundf(__fmul_rn(f[e], id)));
      w[e >> 2] |= (static_cast<uint32_t>(code) & 0xffu) << (8 * (e & 3));
    }
    if (pool != nullptr) {
      uint8_t* t = pool + tile * kQ8TileBytes;
      reinterpret_cast<uint2*>(t)[off * kLanes + c] = make_uint2(w[0], w[1]);
      if ((c & 3) == 0) *reinterpret_cast<__half*>(t + kQ8CodeBytes + (off * 4 + (c >> 2)) * 2) = __float2half_rn(d);
    }
  }
}

template <int kFormat>
__global__ void __launch_bounds__(kRopeThreads) qk_norm_rope_append_kernel(const QkNormRopeArgs a) {
  pdl_wait();  // the projection's output may come from the previous grid
  pdl_trigger();
  const int64_t item = (blockIdx.x * static_cast<int64_t>(kRopeThreads) + threadIdx.x) / kLanes;
  const int c = threadIdx.x & (kLanes - 1);
  const bool live = item < static_cast<int64_t>(a.num_tokens) * a.num_kv_heads;  // uniform over the 16 lanes
  const int64_t t = live ? item / a.num_kv_heads : 0;
  const int h = live ? static_cast<int>(item - t * a.num_kv_heads) : 0;

  // the position first: the table's row waits for it
  const int half = a.rot_dim / 2;
  int pos = half > 0 ? a.positions[t] : 0;
  const int64_t slot = a.slot_mapping[t];
  const uint16_t* qp = static_cast<const uint16_t*>(a.q) + t * a.q_stride + h * (kGroup * kHeadDim) + c * kPerLane;
  const uint16_t* kp = static_cast<const uint16_t*>(a.k) + t * a.k_stride + h * kHeadDim + c * kPerLane;
  const uint16_t* vp = static_cast<const uint16_t*>(a.v) + t * a.v_stride + h * kHeadDim + c * kPerLane;
  uint4 raw[kGroup + 2];
#pragma unroll
  for (int g = 0; g < kGroup; ++g) raw[g] = *reinterpret_cast<const uint4*>(qp + g * kHeadDim);
  raw[kGroup] = *reinterpret_cast<const uint4*>(kp);
  raw[kGroup + 1] = *reinterpret_cast<const uint4*>(vp);
  if (half > 0) {
    if (pos < 0 || pos >= a.max_positions) {
      if (live && c == 0 && h == 0) report(a.err, PKV_DEVERR_POSITION);
      pos = min(max(pos, 0), a.max_positions - 1);
    }
  }
  // cosines and sines of the lane's dims, and the lane that holds their partners
  float cs[kPerLane], sn[kPerLane];
  const int half_lanes = half / kPerLane;
  int src = c;
#pragma unroll
  for (int e = 0; e < kPerLane; ++e) {
    cs[e] = 1.f;
    sn[e] = 0.f;
  }
  if (c < 2 * half_lanes) {
    const float* tab = a.rope_table + static_cast<int64_t>(pos) * a.rot_dim;
    if (a.interleaved) {
      const float4 co = *reinterpret_cast<const float4*>(tab + c * 4);
      const float4 si = *reinterpret_cast<const float4*>(tab + half + c * 4);
      const float cc[4] = {co.x, co.y, co.z, co.w}, ss[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        cs[2 * e] = cs[2 * e + 1] = cc[e];
        sn[2 * e] = -ss[e];
        sn[2 * e + 1] = ss[e];
      }
    } else {
      const bool low = c < half_lanes;
      const int i0 = (low ? c : c - half_lanes) * kPerLane;
      src = low ? c + half_lanes : c - half_lanes;
#pragma unroll
      for (int e = 0; e < kPerLane; e += 4) {
        const float4 co = *reinterpret_cast<const float4*>(tab + i0 + e);
        const float4 si = *reinterpret_cast<const float4*>(tab + half + i0 + e);
        const float sgn = low ? -1.f : 1.f;
        cs[e] = co.x, cs[e + 1] = co.y, cs[e + 2] = co.z, cs[e + 3] = co.w;
        sn[e] = sgn * si.x, sn[e + 1] = sgn * si.y, sn[e + 2] = sgn * si.z, sn[e + 3] = sgn * si.w;
      }
    }
  }

  // the four query heads, then K
  float kf[kPerLane];
#pragma unroll
  for (int g = 0; g < kGroup + 1; ++g) {
    float x[kPerLane];
    unpack8(raw[g], x);
    const uint16_t* wp = static_cast<const uint16_t*>(g < kGroup ? a.q_weight : a.k_weight);
    if (wp != nullptr) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < kPerLane; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
      for (int off = 1; off < kLanes; off <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
      const float rms = rsqrtf(ss * (1.f / kHeadDim) + a.eps);
      float w[kPerLane];
      unpack8(*reinterpret_cast<const uint4*>(wp + c * kPerLane), w);
#pragma unroll
      for (int e = 0; e < kPerLane; ++e) x[e] *= rms * w[e];
    }
    if (half > 0) {
      float y[kPerLane];
      if (a.interleaved) {
#pragma unroll
        for (int e = 0; e < kPerLane; ++e) y[e] = x[e ^ 1];
      } else {
#pragma unroll
        for (int e = 0; e < kPerLane; ++e) y[e] = __shfl_sync(0xffffffffu, x[e], src, kLanes);
      }
      if (c < 2 * half_lanes) {
#pragma unroll
        for (int e = 0; e < kPerLane; ++e) x[e] = fmaf(x[e], cs[e], y[e] * sn[e]);
      }
    }
    if (g < kGroup) {
      if (live)
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.q_out) +
                                  ((t * a.num_kv_heads + h) * kGroup + g) * kHeadDim + c * kPerLane) = pack8(x);
    } else {
#pragma unroll
      for (int e = 0; e < kPerLane; ++e) kf[e] = x[e];
    }
  }

  // K and V into their slot
  const int64_t pool_slots = static_cast<int64_t>(a.num_blocks) * kBlockSize;
  bool store = live && slot >= 0;
  if (store && slot >= pool_slots) {
    if (c == 0 && h == 0) report(a.err, PKV_DEVERR_SLOT);
    store = false;
  }
  const int64_t blk = store ? slot / kBlockSize : 0;
  const int off = store ? static_cast<int>(slot - blk * kBlockSize) : 0;
  const int64_t tile = blk * a.num_kv_heads + h;
  float vf[kPerLane];
  unpack8(raw[kGroup + 1], vf);
  if constexpr (kFormat == PKV_KV_Q8_0) {  // the group maxima are exchanged by whole warps
    store_row<kFormat>(store ? static_cast<uint8_t*>(a.k_cache) : nullptr, tile, off, c, kf);
    store_row<kFormat>(store ? static_cast<uint8_t*>(a.v_cache) : nullptr, tile, off, c, vf);
  } else if (store) {
    store_row<kFormat>(static_cast<uint8_t*>(a.k_cache), tile, off, c, kf);
    store_row<kFormat>(static_cast<uint8_t*>(a.v_cache), tile, off, c, vf);
  }
}

}  // namespace

cudaError_t launch_qk_norm_rope_append(const QkNormRopeArgs& a, int32_t kv_format, cudaStream_t stream) {
  const int64_t threads = static_cast<int64_t>(a.num_tokens) * a.num_kv_heads * kLanes;
  if (threads == 0) return cudaSuccess;
  const int64_t blocks = (threads + kRopeThreads - 1) / kRopeThreads;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(blocks));
  switch (kv_format) {
    case PKV_KV_BF16:
      return launch_pdl(qk_norm_rope_append_kernel<PKV_KV_BF16>, grid, dim3(kRopeThreads), 0, stream, 1, a);
    case PKV_KV_Q8_0:
      return launch_pdl(qk_norm_rope_append_kernel<PKV_KV_Q8_0>, grid, dim3(kRopeThreads), 0, stream, 1, a);
    case PKV_KV_FP8_E4M3:
      return launch_pdl(qk_norm_rope_append_kernel<PKV_KV_FP8_E4M3>, grid, dim3(kRopeThreads), 0, stream, 1, a);
  }
  return cudaErrorInvalidValue;
}

}  // namespace pkv
