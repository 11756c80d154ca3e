// kv_append_scaled.cu -- store new tokens in a paged KV cache of E4M3 codes
// with one FP32 scale for each block of 16 tokens and KV head ("Chapter 8:
// Inference Optimization", clxhxhhr.top/posts/4341, §8.4.4: K and V in FP8;
// §8.4.2: values that lie together share a scale).
//
// Mathematics: value = code * scale.  A scale is a power of two, the smallest
// of 2^-32 .. 2^32 under which the block's largest magnitude is at most 448:
// codes are floating point, so a scale between two powers of two would gain
// nothing but the last binade, and a power of two divides exactly.  A block
// that already holds tokens keeps its scale unless the new ones need a larger
// one; then its codes are divided by the ratio, exactly but where they leave
// E4M3's normal range (2^-6), and rounded to nearest there.  A block's first
// token starts it anew, whatever it held.
//
// One warp owns a (block, KV head) of the call, K and V, so nothing is shared:
// 16 lanes a token of 16 bytes, up to 16 loads in flight, the largest magnitude
// by one reduction over BF16 bits (their order is that of integers).  Bound by
// HBM for prompts and by a chain of four dependent reads (request, context,
// block, its scale) for single tokens.  Measured, 8 KV heads: 4 prompts of 8100
// to 8192 tokens 37 us (5.4 TB/s), 24 chunks of 5 to 700 7 us, one token each of
// 37 requests 2.8 us from a graph.  (Prompts with 2, 4 or 8 warps a CTA: no faster.)
#include "pkv_common.cuh"
#include "pkv_kernels.h"

namespace pkv {
namespace {

constexpr int kAsWarps = 1;
constexpr int kAsLowest = -32, kAsHighest = 32;  // exponents of the scales

// 4 BF16 values (two words) times `f`, as E4M3 bytes (nearest even, saturating).
__device__ __forceinline__ uint32_t as_codes(uint32_t w0, uint32_t w1, float f) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(bf16_hi(w0) * f), "f"(bf16_lo(w0) * f));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(bf16_hi(w1) * f), "f"(bf16_lo(w1) * f));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// The same, divided by a scale that is no power of two.
__device__ __forceinline__ uint32_t as_codes_div(uint32_t w0, uint32_t w1, float s) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
      : "=h"(lo)
      : "f"(__fdiv_rn(bf16_hi(w0), s)), "f"(__fdiv_rn(bf16_lo(w0), s)));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
      : "=h"(hi)
      : "f"(__fdiv_rn(bf16_hi(w1), s)), "f"(__fdiv_rn(bf16_lo(w1), s)));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// 4 E4M3 codes times `f` (at most 1), rounded to E4M3 again.
__device__ __forceinline__ uint32_t as_rescale(uint32_t codes, float f) {
  uint32_t out = 0;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    uint32_t h2;
    const uint16_t pair = static_cast<uint16_t>(codes >> (16 * k));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(pair));
    float lo, hi;
    asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(h2));
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi * f), "f"(lo * f));
    out |= static_cast<uint32_t>(r) << (16 * k);
  }
  return out;
}

// Places: request r's blocks have the places first_place(r) .. : a request of
// n new tokens touches at most n / 16 + 2 blocks, which is no more than the
// distance to the next request's first place.  (Where cu_new falls, places no
// longer rise with the requests, and some find another request than theirs: their
// blocks are left out, which the report of the wrong entry stands for.  With a
// check of all entries by each warp, to refuse the call: 64 requests of up to 200
// tokens 9.6 us, not 9.2, 300 of one 7.8, not 6.8, 4096 of one 147, not 105.)
__device__ __forceinline__ int64_t first_place(const AppendScaledArgs& a, int r) {
  return a.cu_new == nullptr ? r : (int64_t{max(a.cu_new[r], 0)} >> 4) + 2 * int64_t{r};
}

__global__ void __launch_bounds__(kAsWarps * 32) kv_append_scaled_kernel(const AppendScaledArgs a, int64_t items) {
  pdl_wait();  // new K/V, tables and lengths may come from the previous grid
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * kAsWarps;
  if (a.cu_new != nullptr && blockIdx.x == gridDim.x - 1 && threadIdx.x < 32) {
    bool bad = false;
    for (int s = lane; s < a.num_seqs; s += 32)
      bad = bad || a.cu_new[s] < 0 || a.cu_new[s + 1] < a.cu_new[s] || a.cu_new[s + 1] > a.num_tokens;
    if (bad) report(a.err, PKV_DEVERR_SEQLENS);
  }
  for (int64_t item = static_cast<int64_t>(blockIdx.x) * kAsWarps + (threadIdx.x >> 5); item < items; item += warps) {
    // item = place * Hkv + h
    const int64_t place = item / a.num_kv_heads;
    const int h = static_cast<int>(item - place * a.num_kv_heads);
    int r;
    if (a.cu_new == nullptr) {
      r = static_cast<int>(place);
    } else {  // the last request whose first place is not behind this one, 32 ways at a time
      int lo = 0, hi = a.num_seqs;  // in [lo, hi)
      while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int x = lo + lane * step;
        const uint32_t in = __ballot_sync(0xffffffffu, x < hi && first_place(a, x) <= place);
        const int last = in == 0 ? 0 : 31 - __clz(in);
        lo += last * step;
        hi = min(hi, lo + step);
      }
      r = lo;
    }
    const bool once = lane == 0 && h == 0;
    const int64_t nth = place - first_place(a, r);  // of the request's touched blocks
    const int t0 = a.cu_new == nullptr ? r : a.cu_new[r];
    const int t1 = a.cu_new == nullptr ? r + 1 : a.cu_new[r + 1];
    if (t0 < 0 || t1 < t0 || t1 > a.num_tokens) continue;  // (reported above)
    const int ctx = a.context_lens[r];
    const int n = t1 - t0;
    if (n == 0 || ctx <= 0) continue;  // nothing new, or a padding row
    if (ctx < n || ctx > a.max_blocks * kBlockSize) {
      if (once && nth == 0) report(a.err, PKV_DEVERR_CONTEXT);
      continue;
    }
    const int p0 = ctx - n;  // position of the request's first new token
    const int64_t lb = p0 / kBlockSize + nth;
    if (nth < 0 || lb > (ctx - 1) / kBlockSize) continue;
    const int32_t blk = a.block_tables[static_cast<int64_t>(r) * a.max_blocks + lb];
    const int first = max(p0 - static_cast<int>(lb) * kBlockSize, 0);          // offsets [first, end) are new,
    const int end = min(ctx - static_cast<int>(lb) * kBlockSize, kBlockSize);  // [0, first) hold tokens
    const int tok = t0 + static_cast<int>(lb) * kBlockSize + first - p0;       // the token at offset `first`
    // lane l: 8 values of the tokens first + l / 16, + 2, + 4, ...
    const int half = lane >> 4;
    const int64_t in_row = static_cast<int64_t>(h) * kHeadDim + (lane & 15) * 8;
    uint4 w[2][8];  // K, V
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const int64_t stride = which ? a.v_stride : a.k_stride;
      const uint16_t* src = (which ? a.v_new : a.k_new) + (static_cast<int64_t>(tok) + half) * stride + in_row;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        w[which][k] = make_uint4(0, 0, 0, 0);
        if (first + 2 * k + half < end) w[which][k] = *reinterpret_cast<const uint4*>(src + 2 * k * stride);
      }
    }
    if (blk < 0 || blk >= a.num_blocks) {
      if (once) report(a.err, PKV_DEVERR_BLOCK_ID);
      continue;
    }
    const int64_t at = static_cast<int64_t>(blk) * a.num_kv_heads + h;
    float old[2] = {0.f, 0.f};
    if (first > 0) {
      old[0] = a.k_scales[at];
      old[1] = a.v_scales[at];
    }
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      uint32_t top = 0;  // pairs of magnitudes
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint4 x = w[which][k];
        top = __vmaxu2(__vmaxu2(top, x.x & 0x7fff7fffu), x.y & 0x7fff7fffu);
        top = __vmaxu2(__vmaxu2(top, x.z & 0x7fff7fffu), x.w & 0x7fff7fffu);
      }
      top = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
      // 448 = 1.75 * 2^8: the exponent field less (127 + 8), one more above 1.75
      int e = static_cast<int>(top >> 7) - 135 + ((top & 0x7fu) > 0x60u ? 1 : 0);
      e = min(max(e, kAsLowest), kAsHighest);
      const float need = __int_as_float((127 + e) << 23);
      const float scale = fmaxf(old[which], need);
      uint8_t* tile = (which ? a.v_cache : a.k_cache) + at * kFp8TileBytes + (lane & 15) * 8;
      const bool power = (__float_as_uint(scale) & 0x7fffffu) == 0;
      const float inv = 1.f / scale;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int off = first + 2 * k + half;
        if (off < end) {
          const uint4 x = w[which][k];
          uint2 c;
          if (power) {
            c = make_uint2(as_codes(x.x, x.y, inv), as_codes(x.z, x.w, inv));
          } else {
            c = make_uint2(as_codes_div(x.x, x.y, scale), as_codes_div(x.z, x.w, scale));
          }
          *reinterpret_cast<uint2*>(tile + off * kHeadDim) = c;
        }
      }
      if (first > 0 && scale > old[which]) {  // the earlier tokens follow the scale
        const float f = __fdiv_rn(old[which], scale);
        for (int off = half; off < first; off += 2) {
          uint2* p = reinterpret_cast<uint2*>(tile + off * kHeadDim);
          const uint2 c = *p;
          *p = make_uint2(as_rescale(c.x, f), as_rescale(c.y, f));
        }
      }
      if (lane == 0 && scale != old[which]) (which ? a.v_scales : a.k_scales)[at] = scale;
    }
  }
}

// A CTA moves one block of one tensor with its scales.
__global__ void __launch_bounds__(256)
    copy_blocks_scaled_kernel(uint8_t* k_cache, uint8_t* v_cache, float* k_scales, float* v_scales, int32_t num_blocks,
                              int32_t num_kv_heads, const int32_t* __restrict__ src, const int32_t* __restrict__ dst,
                              unsigned int* err) {
  pdl_wait();
  pdl_trigger();
  const int pair = blockIdx.x >> 1;
  const int32_t s = src[pair], d = dst[pair];
  if (s < 0 || s >= num_blocks || d < 0 || d >= num_blocks) {
    if (threadIdx.x == 0) report(err, PKV_DEVERR_BLOCK_ID);
    return;
  }
  uint8_t* cache = (blockIdx.x & 1) ? v_cache : k_cache;
  float* scales = (blockIdx.x & 1) ? v_scales : k_scales;
  const int64_t bytes = static_cast<int64_t>(num_kv_heads) * kFp8TileBytes;
  const uint4* from = reinterpret_cast<const uint4*>(cache + s * bytes);
  uint4* to = reinterpret_cast<uint4*>(cache + d * bytes);
  for (int64_t i = threadIdx.x; i < bytes / 16; i += blockDim.x) to[i] = from[i];
  for (int i = threadIdx.x; i < num_kv_heads; i += blockDim.x)
    scales[static_cast<int64_t>(d) * num_kv_heads + i] = scales[static_cast<int64_t>(s) * num_kv_heads + i];
}

}  // namespace

cudaError_t launch_kv_append_scaled(const AppendScaledArgs& a, cudaStream_t stream) {
  const int64_t places =
      a.cu_new == nullptr ? a.num_seqs : static_cast<int64_t>(a.num_tokens) / kBlockSize + 2 * static_cast<int64_t>(a.num_seqs);
  const int64_t items = places * a.num_kv_heads;
  int64_t blocks = (items + kAsWarps - 1) / kAsWarps;
  if (blocks > 1 << 20) blocks = 1 << 20;
  return launch_pdl(kv_append_scaled_kernel, dim3(static_cast<unsigned>(blocks)), dim3(kAsWarps * 32), 0, stream, 1, a,
                    items);
}

cudaError_t launch_copy_blocks_scaled(uint8_t* k_cache, uint8_t* v_cache, float* k_scales, float* v_scales,
                                      int32_t num_blocks, int32_t num_kv_heads, const int32_t* src,
                                      const int32_t* dst, int32_t num_pairs, unsigned int* err, cudaStream_t stream) {
  return launch_pdl(copy_blocks_scaled_kernel, dim3(static_cast<unsigned>(num_pairs) * 2), dim3(256), 0, stream, 1,
                    k_cache, v_cache, k_scales, v_scales, num_blocks, num_kv_heads, src, dst, err);
}

}  // namespace pkv
