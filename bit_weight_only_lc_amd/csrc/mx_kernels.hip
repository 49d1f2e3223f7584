// Block-scaled storage of activations and weights, and the SiLU gate that keeps its
// operands in it. All of these read and write each value once and are bound by HBM: bf16 at
// 8192 x 11008, gate forward with three checkpoints 139 us (0.82 GB, 5.9 TB/s), backward
// 132 us (0.73 GB, 5.5 TB/s), MXINT8 quantisation of 8192 x 14336 69 us (0.36 GB, 5.1 TB/s);
// a copy of 1 GiB reaches 5.2 TB/s, of 256 MiB 5.5.
// Rows are made of whole blocks of 32, so a matrix is a flat run of blocks; a lane takes 8
// consecutive values and four lanes share a block.
#include "mx_device.h"
#include "lcvq_internal.h"

namespace lcvq {

// ------------------------------------------------------------------ quantise, dequantise
template <typename T, int FMT>
__global__ __launch_bounds__(256) void k_mx_quantize(const T* __restrict__ X, int64_t groups,
                                                     void* __restrict__ codes,
                                                     uint8_t* __restrict__ scales) {
  const int64_t step = (int64_t)gridDim.x * 256;
  for (int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x; g < groups; g += step) {
    float v[8];
    load8(X + g * 8, v);
    const uint32_t byte = mx_block_byte<FMT>(v);
    if constexpr (FMT == MX_FP4)
      static_cast<uint32_t*>(codes)[g] = mx_encode_fp4(v, byte);
    else
      static_cast<uint2*>(codes)[g] = mx_encode_int8(v, byte);
    if ((g & 3) == 0) scales[g >> 2] = (uint8_t)byte;
  }
}

template <typename T, int FMT>
__global__ __launch_bounds__(256) void k_mx_dequantize(const void* __restrict__ codes,
                                                       const uint8_t* __restrict__ scales,
                                                       int64_t groups, T* __restrict__ out) {
  const int64_t step = (int64_t)gridDim.x * 256;
  for (int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x; g < groups; g += step) {
    float v[8];
    if constexpr (FMT == MX_FP4)
      mx_decode_fp4(static_cast<const uint32_t*>(codes)[g], scales[g >> 2], v);
    else
      mx_decode_int8(static_cast<const uint2*>(codes)[g], scales[g >> 2], v);
    store8(out + g * 8, v);
  }
}

// ------------------------------------------------------------------ SiLU gate
// s = 1 / (1 + e^-g) and 1 - s = e^-g s, which loses nothing where s is near 1. The hardware's
// reciprocal and one Newton step: without the step H rounds to another bf16 now and then, and
// an IEEE division is no longer hidden by the loads (forward 144 -> 167 us at 8192 x 11008).
// Below -80, where e^-g overflows in the end, s = e^g to the last bit; a thread's values are
// tested for that together.
__device__ __forceinline__ void sigmoid8(const float (&g)[8], float (&s)[8], float (&one_minus_s)[8]) {
  float low = g[0];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float e = expf(-fmaxf(g[j], -80.f));
    const float q = 1.f + e, r = __builtin_amdgcn_rcpf(q);
    s[j] = __builtin_fmaf(__builtin_fmaf(-q, r, 1.f), r, r);
    one_minus_s[j] = e * s[j];
    low = fminf(low, g[j]);
  }
  if (__builtin_expect(low < -80.f, 0)) {
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] = g[j] < -80.f ? expf(g[j]) : s[j];
  }
}

struct GateCkpt {
  uint2* c;                  // MXINT8 codes, 8 per group
  uint8_t* s;                // scale bytes
};
__device__ __forceinline__ void ckpt_store(const GateCkpt& k, int64_t g, const float (&v)[8]) {
  const uint32_t byte = mx_block_byte<MX_INT8>(v);
  k.c[g] = mx_encode_int8(v, byte);
  if ((g & 3) == 0) k.s[g >> 2] = (uint8_t)byte;
}

__device__ __forceinline__ float as_written(uint16_t*, float x) {
  return bf16lo_to_f32(pack_bf16x2(x, 0.f));
}
__device__ __forceinline__ float as_written(float*, float x) { return x; }

template <typename T>
__global__ __launch_bounds__(256) void k_silu_gate_fwd(const T* __restrict__ G,
                                                       const T* __restrict__ U, int64_t groups,
                                                       T* __restrict__ H, GateCkpt gk,
                                                       GateCkpt uk, GateCkpt hk) {
  const int64_t step = (int64_t)gridDim.x * 256;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < groups; i += step) {
    float g[8], u[8], h[8];
    load8(G + i * 8, g);
    load8(U + i * 8, u);
    float s[8], r[8];
    sigmoid8(g, s, r);
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = as_written(H, g[j] * s[j] * u[j]);
    store8(H + i * 8, h);
    if (gk.c) ckpt_store(gk, i, g);
    if (uk.c) ckpt_store(uk, i, u);
    if (hk.c) ckpt_store(hk, i, h);
  }
}

template <typename T>
__global__ __launch_bounds__(256) void k_silu_gate_bwd(const T* __restrict__ dH, int64_t groups,
                                                       const uint2* __restrict__ Gc,
                                                       const uint8_t* __restrict__ Gs,
                                                       const uint2* __restrict__ Uc,
                                                       const uint8_t* __restrict__ Us,
                                                       T* __restrict__ dG, T* __restrict__ dU) {
  const int64_t step = (int64_t)gridDim.x * 256;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < groups; i += step) {
    float g[8], u[8], d[8], a[8], b[8];
    load8(dH + i * 8, d);
    mx_decode_int8(Gc[i], Gs[i >> 2], g);
    mx_decode_int8(Uc[i], Us[i >> 2], u);
    float s[8], r[8];
    sigmoid8(g, s, r);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      b[j] = d[j] * (g[j] * s[j]);
      a[j] = d[j] * u[j] * (s[j] * (1.f + g[j] * r[j]));
    }
    store8(dG + i * 8, a);
    store8(dU + i * 8, b);
  }
}

// ------------------------------------------------------------------ launchers
static dim3 flat_grid(int64_t groups) {
  int64_t b = (groups + 255) / 256;
  if (b > 65535) b = 65535;
  return dim3((unsigned)(b < 1 ? 1 : b));
}

hipError_t launch_mx_quantize(const void* X, bool f32, int64_t n, int fmt, void* codes,
                              uint8_t* scales, hipStream_t s) {
  const int64_t groups = n / 8;
  const dim3 g = flat_grid(groups), b(256);
  const float* xf = static_cast<const float*>(X);
  const uint16_t* xh = static_cast<const uint16_t*>(X);
  if (f32 && fmt == MX_FP4)
    hipLaunchKernelGGL((k_mx_quantize<float, MX_FP4>), g, b, 0, s, xf, groups, codes, scales);
  else if (f32)
    hipLaunchKernelGGL((k_mx_quantize<float, MX_INT8>), g, b, 0, s, xf, groups, codes, scales);
  else if (fmt == MX_FP4)
    hipLaunchKernelGGL((k_mx_quantize<uint16_t, MX_FP4>), g, b, 0, s, xh, groups, codes, scales);
  else
    hipLaunchKernelGGL((k_mx_quantize<uint16_t, MX_INT8>), g, b, 0, s, xh, groups, codes, scales);
  return hipGetLastError();
}

hipError_t launch_mx_dequantize(const void* codes, const uint8_t* scales, int64_t n, int fmt,
                                void* out, bool f32, hipStream_t s) {
  const int64_t groups = n / 8;
  const dim3 g = flat_grid(groups), b(256);
  float* of = static_cast<float*>(out);
  uint16_t* oh = static_cast<uint16_t*>(out);
  if (f32 && fmt == MX_FP4)
    hipLaunchKernelGGL((k_mx_dequantize<float, MX_FP4>), g, b, 0, s, codes, scales, groups, of);
  else if (f32)
    hipLaunchKernelGGL((k_mx_dequantize<float, MX_INT8>), g, b, 0, s, codes, scales, groups, of);
  else if (fmt == MX_FP4)
    hipLaunchKernelGGL((k_mx_dequantize<uint16_t, MX_FP4>), g, b, 0, s, codes, scales, groups, oh);
  else
    hipLaunchKernelGGL((k_mx_dequantize<uint16_t, MX_INT8>), g, b, 0, s, codes, scales, groups, oh);
  return hipGetLastError();
}

hipError_t launch_silu_gate_fwd(const void* G, const void* U, bool f32, int64_t n, void* H,
                                int8_t* Gc, uint8_t* Gs, int8_t* Uc, uint8_t* Us, int8_t* Hc,
                                uint8_t* Hs, hipStream_t s) {
  const int64_t groups = n / 8;
  const dim3 g = flat_grid(groups), b(256);
  const GateCkpt gk{reinterpret_cast<uint2*>(Gc), Gs}, uk{reinterpret_cast<uint2*>(Uc), Us},
      hk{reinterpret_cast<uint2*>(Hc), Hs};
  if (f32)
    hipLaunchKernelGGL(k_silu_gate_fwd<float>, g, b, 0, s, static_cast<const float*>(G),
                       static_cast<const float*>(U), groups, static_cast<float*>(H), gk, uk, hk);
  else
    hipLaunchKernelGGL(k_silu_gate_fwd<uint16_t>, g, b, 0, s, static_cast<const uint16_t*>(G),
                       static_cast<const uint16_t*>(U), groups, static_cast<uint16_t*>(H), gk,
                       uk, hk);
  return hipGetLastError();
}

hipError_t launch_silu_gate_bwd(const void* dH, bool f32, int64_t n, const int8_t* Gc,
                                const uint8_t* Gs, const int8_t* Uc, const uint8_t* Us, void* dG,
                                void* dU, hipStream_t s) {
  const int64_t groups = n / 8;
  const dim3 g = flat_grid(groups), b(256);
  const uint2* gc = reinterpret_cast<const uint2*>(Gc);
  const uint2* uc = reinterpret_cast<const uint2*>(Uc);
  if (f32)
    hipLaunchKernelGGL(k_silu_gate_bwd<float>, g, b, 0, s, static_cast<const float*>(dH), groups,
                       gc, Gs, uc, Us, static_cast<float*>(dG), static_cast<float*>(dU));
  else
    hipLaunchKernelGGL(k_silu_gate_bwd<uint16_t>, g, b, 0, s, static_cast<const uint16_t*>(dH),
                       groups, gc, Gs, uc, Us, static_cast<uint16_t*>(dG),
                       static_cast<uint16_t*>(dU));
  return hipGetLastError();
}

}  // namespace lcvq
