// prism_ckpt8_pack / prism_ckpt8_unpack: 8-bit checkpoints of activations
// (format and arithmetic: ckpt8.cuh), for tensors that a training step keeps
// between its forward and its backward.
//
// HBM-bound, one pass: pack reads 2 bytes and writes 33/32 bytes per value,
// unpack the reverse.  Sixteen lanes own 128 channels of a row (a group): each
// lane holds eight (one 16-byte vector), four lanes share a block's maximum by
// shuffles, and lane 0 of the sixteen writes their four scales as one word.
// What had to go to reach the memory's rate was integer work: rows are found by
// stepping (one division per thread), the maximum is taken on pairs of bf16 bits.
#include <algorithm>
#include <cstdio>

#include "ckpt8.cuh"
#include "internal.h"

namespace prism {
namespace ck8 {

constexpr int kThreads = 256;
// 128-channel groups in flight per half-warp, and CTAs per SM of a full grid.
// 24 (three waves) beats one resident wave of 8: CTAs then start and end apart
// from one another.  Measured over 276480 x 1024: unpack 151.6 -> 139.4 us, pack
// 163.8 -> 153.9; pack with two groups instead of four 144.2, unpack 164.4.
constexpr int kPackUnroll = 2, kUnpackUnroll = 4, kCtasPerSm = 24;

// vec: 16-byte vectors of a row that exist (the rest of the last group is zero)
__global__ void __launch_bounds__(kThreads)
    pack_kernel(const uint4 *__restrict__ x, long long ld_vec, int vec, const Walk w, uint2 *__restrict__ codes,
                uint32_t *__restrict__ scales) {
  const int l16 = threadIdx.x & 15;
  Place p(w, ((long long)blockIdx.x * kThreads + threadIdx.x) >> 4);
  // both half-warps of a warp run the same number of iterations (shuffles)
  while (__any_sync(0xffffffffu, p.g < w.groups)) {
    uint4 in[kPackUnroll];
    long long g[kPackUnroll];
#pragma unroll
    for (int u = 0; u < kPackUnroll; ++u) {
      const int c = p.col * 16 + l16;
      g[u] = p.g;
      in[u] = make_uint4(0, 0, 0, 0);
      if (p.g < w.groups && c < vec) in[u] = __ldcs(x + p.row * ld_vec + c);
      p.step(w);
    }
#pragma unroll
    for (int u = 0; u < kPackUnroll; ++u) {
      const uint32_t h[4] = {in[u].x, in[u].y, in[u].z, in[u].w};
      // magnitudes of the pairs; a NaN's bits compare above infinity's
      uint32_t m = __vmaxu2(__vmaxu2(h[0] & 0x7fff7fffu, h[1] & 0x7fff7fffu), __vmaxu2(h[2] & 0x7fff7fffu, h[3] & 0x7fff7fffu));
      m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const uint32_t top = max(m << 16, m & 0xffff0000u);
      const uint32_t s = ckpt8_scale(top);
      const float inv = ckpt8_inverse(s);
      float v[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[2 * k] = bf16lo(h[k]);
        v[2 * k + 1] = bf16hi(h[k]);
      }
      if (top > kCkptTop) {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = s == kCkptBad ? 0.f : ckpt8_clamp(v[k]);
      }
      uint32_t sw = s << (8 * (l16 >> 2));
      sw |= __shfl_xor_sync(0xffffffffu, sw, 4);
      sw |= __shfl_xor_sync(0xffffffffu, sw, 8);
      if (g[u] < w.groups) {
        __stcs(codes + g[u] * 16 + l16,
               make_uint2(ckpt8_code4(v[0], v[1], v[2], v[3], inv), ckpt8_code4(v[4], v[5], v[6], v[7], inv)));
        if (l16 == 0) scales[g[u]] = sw;
      }
    }
  }
}

__global__ void __launch_bounds__(kThreads)
    unpack_kernel(const uint2 *__restrict__ codes, const uint8_t *__restrict__ scales, const Walk w, int vec,
                  uint4 *__restrict__ x, long long ld_vec) {
  unpack_walk<kUnpackUnroll>(codes, scales, w, vec, x, ld_vec, ((long long)blockIdx.x * kThreads + threadIdx.x) >> 4);
}

// one iteration of `unroll` groups per half-warp, or full occupancy
Walk walk_for(long long n, long long ld, int unroll, int &grid) {
  const long long per_cta = (long long)(kThreads / 16) * unroll;
  grid = (int)std::min<long long>((n * (ld / 128) + per_cta - 1) / per_cta, (long long)device_sm_count() * kCtasPerSm);
  return make_walk(n, ld, (long long)grid * (kThreads / 16));
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
  if (!bad) {
    const Span codes("the codes", c->codes, 1, n * c->ld), scales("the scales", c->scales, 1, n * c->ld / 32);
    const Span v("the activation", x, n, 2 * (uint64_t)width, 2 * (uint64_t)ld);
    if (overlap(v, codes) || overlap(v, scales)) bad = "the activation overlaps the checkpoint";
    else if (overlap(codes, scales)) bad = "the codes overlap the scales";
  }
  if (!bad) return PRISM_OK;
  snprintf(msg, sizeof(msg), "%s: %s", who, bad);
  return report_error(PRISM_ERR_INVALID_ARG, msg);
}

int finish(const char *who, cudaError_t e) {
  if (e != cudaSuccess) {
    char msg[256];
    snprintf(msg, sizeof(msg), "%s: %s", who, cudaGetErrorString(e));
    return report_error(PRISM_ERR_CUDA, msg);
  }
  clear_error();
  return PRISM_OK;
}

}  // namespace ck8

cudaError_t launch_ckpt8_unpack(const prism_ckpt8_t &in, long long n, int width, uint16_t *x, long long ld,
                                cudaStream_t st) {
  int grid;
  const Walk w = ck8::walk_for(n, in.ld, ck8::kUnpackUnroll, grid);
  ck8::unpack_kernel<<<grid, ck8::kThreads, 0, st>>>(reinterpret_cast<const uint2 *>(in.codes), in.scales, w, width / 8,
                                                     reinterpret_cast<uint4 *>(x), ld / 8);
  count_launches(1);
  return cudaGetLastError();
}

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
  int grid;
  const Walk w = ck8::walk_for(n, out->ld, ck8::kPackUnroll, grid);
  ck8::pack_kernel<<<grid, ck8::kThreads, 0, st>>>(reinterpret_cast<const uint4 *>(x), (long long)(ld / 8), width / 8, w,
                                                   reinterpret_cast<uint2 *>(out->codes),
                                                   reinterpret_cast<uint32_t *>(out->scales));
  count_launches(1);
  return ck8::finish("prism_ckpt8_pack", cudaGetLastError());
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
  return ck8::finish("prism_ckpt8_unpack", launch_ckpt8_unpack(*in, n, width, x, ld, reinterpret_cast<cudaStream_t>(stream)));
}
