// prism_ckpt8_pack / prism_ckpt8_unpack: 8-bit checkpoints of activations
// (format and arithmetic: ckpt8.cuh), for tensors that a training step keeps
// between its forward and its backward.
//
// HBM-bound, one pass: pack reads 2 bytes and writes 33/32 bytes per value,
// unpack the reverse.  Sixteen lanes own 128 channels of a row: each lane holds
// eight (one 16-byte vector), four lanes share a block's maximum by shuffles,
// and lane 0 of the sixteen writes their four scales as one word.
#include <algorithm>
#include <cstdio>

#include "ckpt8.cuh"
#include "internal.h"

namespace prism {
namespace ck8 {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;  // 128-channel groups in flight per half-warp

__device__ __forceinline__ void unpack8(const uint4 &x, float (&v)[8]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    v[2 * k] = bf16lo(w[k]);
    v[2 * k + 1] = bf16hi(w[k]);
  }
}

// groups: n * gpr groups of 128 channels, row-major; vec: 16-byte vectors of a
// row that exist (the rest of the last group is zero)
__global__ void __launch_bounds__(kThreads)
    pack_kernel(const uint4 *__restrict__ x, long long ld_vec, int vec, long long groups, int gpr,
                uint2 *__restrict__ codes, uint32_t *__restrict__ scales) {
  const int l16 = threadIdx.x & 15;
  const long long half = ((long long)blockIdx.x * kThreads + threadIdx.x) >> 4;
  const long long nhalf = ((long long)gridDim.x * kThreads) >> 4;
  // both half-warps of a warp run the same number of iterations (shuffles)
  for (long long g0 = half & ~1LL; g0 < groups; g0 += nhalf * kUnroll) {
    uint4 in[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const long long g = g0 + (half & 1) + u * nhalf;
      in[u] = make_uint4(0, 0, 0, 0);
      if (g < groups) {
        const long long row = g / gpr;
        const int c = (int)(g - row * gpr) * 16 + l16;
        if (c < vec) in[u] = __ldcs(x + row * ld_vec + c);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const long long g = g0 + (half & 1) + u * nhalf;
      float v[8];
      unpack8(in[u], v);
      uint32_t top = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) top = max(top, __float_as_uint(v[k]) & 0x7fffffffu);
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const uint32_t s = ckpt8_scale(top);
      const float inv = ckpt8_inverse(s);
      if (top > kCkptTop) {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = s == kCkptBad ? 0.f : ckpt8_clamp(v[k]);
      }
      uint32_t sw = s << (8 * (l16 >> 2));
      sw |= __shfl_xor_sync(0xffffffffu, sw, 4);
      sw |= __shfl_xor_sync(0xffffffffu, sw, 8);
      if (g < groups) {
        codes[g * 16 + l16] =
            make_uint2(ckpt8_code4(v[0], v[1], v[2], v[3], inv), ckpt8_code4(v[4], v[5], v[6], v[7], inv));
        if (l16 == 0) scales[g] = sw;
      }
    }
  }
}

__global__ void __launch_bounds__(kThreads)
    unpack_kernel(const uint2 *__restrict__ codes, const uint8_t *__restrict__ scales, long long groups, int gpr,
                  int vec, uint4 *__restrict__ x, long long ld_vec) {
  const int l16 = threadIdx.x & 15;
  const long long half = ((long long)blockIdx.x * kThreads + threadIdx.x) >> 4;
  const long long nhalf = ((long long)gridDim.x * kThreads) >> 4;
  for (long long g0 = half; g0 < groups; g0 += nhalf * kUnroll) {
    uint2 q[kUnroll];
    uint32_t s[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const long long g = g0 + u * nhalf;
      if (g < groups) {
        q[u] = __ldcs(codes + g * 16 + l16);
        s[u] = __ldcs(scales + g * 4 + (l16 >> 2));
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const long long g = g0 + u * nhalf;
      if (g >= groups) break;
      const long long row = g / gpr;
      const int c = (int)(g - row * gpr) * 16 + l16;
      const uint32_t s2 = ckpt8_scale2(s[u]);
      if (c < vec)
        __stcs(x + row * ld_vec + c,
               make_uint4(ckpt8_restore2(q[u].x, 0x4140, s2), ckpt8_restore2(q[u].x, 0x4342, s2),
                          ckpt8_restore2(q[u].y, 0x4140, s2), ckpt8_restore2(q[u].y, 0x4342, s2)));
    }
  }
}

// one iteration of kUnroll groups per half-warp, or full occupancy
int grid_for(long long groups) {
  const long long per_cta = (long long)(kThreads / 16) * kUnroll;
  return (int)std::min<long long>((groups + per_cta - 1) / per_cta, (long long)device_sm_count() * 8);
}

int check(const char *who, const uint16_t *x, int64_t n, int32_t width, int64_t ld, const prism_ckpt8_t *c) {
  char msg[200];
  const char *bad = nullptr;
  if (n < 0 || n >= (1LL << 31)) bad = "n must be in [0, 2^31)";
  else if (width <= 0 || width % 8 || width > (1 << 20)) bad = "width must be a positive multiple of 8, <= 2^20";
  else if (ld < width || ld % 8) bad = "ld must be a multiple of 8 and >= width";
  else if (!c) bad = "the checkpoint is NULL";
  else if (c->ld < width || c->ld % 128) bad = "the checkpoint's ld must be a multiple of 128 and >= width";
  else if (c->ld - width >= 128) bad = "the checkpoint's ld must be width rounded up to a multiple of 128";
  else if (n > 0 && (!x || !c->codes || !c->scales)) bad = "NULL pointer";
  else if (reinterpret_cast<uintptr_t>(x) % 16 || reinterpret_cast<uintptr_t>(c->codes) % 16 ||
           reinterpret_cast<uintptr_t>(c->scales) % 4)
    bad = "the activation and the codes must be 16-byte aligned, the scales 4-byte";
  if (!bad) return PRISM_OK;
  snprintf(msg, sizeof(msg), "%s: %s", who, bad);
  return report_error(PRISM_ERR_INVALID_ARG, msg);
}

int finish(const char *who) {
  count_launches(1);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    char msg[256];
    snprintf(msg, sizeof(msg), "%s: %s", who, cudaGetErrorString(e));
    return report_error(PRISM_ERR_CUDA, msg);
  }
  clear_error();
  return PRISM_OK;
}

}  // namespace ck8
}  // namespace prism

using namespace prism;

extern "C" int prism_ckpt8_pack(const uint16_t *x, int64_t n, int32_t width, int64_t ld, const prism_ckpt8_t *out,
                                prism_stream_t stream) {
  NvtxRange nvtx_("prism_ckpt8_pack");
  const int rc = ck8::check("prism_ckpt8_pack", x, n, width, ld, out);
  if (rc != PRISM_OK) return rc;
  if (n == 0) {
    clear_error();
    return PRISM_OK;
  }
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int gpr = (int)(out->ld / 128);
  const long long groups = (long long)n * gpr;
  ck8::pack_kernel<<<ck8::grid_for(groups), ck8::kThreads, 0, st>>>(
      reinterpret_cast<const uint4 *>(x), (long long)(ld / 8), width / 8, groups, gpr,
      reinterpret_cast<uint2 *>(out->codes), reinterpret_cast<uint32_t *>(out->scales));
  return ck8::finish("prism_ckpt8_pack");
}

extern "C" int prism_ckpt8_unpack(const prism_ckpt8_t *in, int64_t n, int32_t width, uint16_t *x, int64_t ld,
                                  prism_stream_t stream) {
  NvtxRange nvtx_("prism_ckpt8_unpack");
  const int rc = ck8::check("prism_ckpt8_unpack", x, n, width, ld, in);
  if (rc != PRISM_OK) return rc;
  if (n == 0) {
    clear_error();
    return PRISM_OK;
  }
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int gpr = (int)(in->ld / 128);
  const long long groups = (long long)n * gpr;
  ck8::unpack_kernel<<<ck8::grid_for(groups), ck8::kThreads, 0, st>>>(
      reinterpret_cast<const uint2 *>(in->codes), in->scales, groups, gpr, width / 8, reinterpret_cast<uint4 *>(x),
      (long long)(ld / 8));
  return ck8::finish("prism_ckpt8_unpack");
}
