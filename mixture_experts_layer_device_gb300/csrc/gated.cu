// The elementwise step of the gated products' backward:
//   dg = dh u act'(g),  du = dh act(g)
// from dh [rows, m] and the saved [g | u] [rows, 2m] to [dg | du], the operand of the
// two products that follow (grouped.cu, grouped_tc.cu), rounded to their 16 bits.
// Bound by memory: ten bytes per element of h.
#include "block.h"
#include "elem.cuh"
#include "gate_act.cuh"
#include "kernels.h"

namespace moe {

namespace {

template <typename T, int ACT>
__global__ void __launch_bounds__(256) gated_slope_kernel(const GatedArgs a, bool vec) {
  const int chunks = (a.m + 7) >> 3;
  const long total = static_cast<long>(a.rows) * chunks;
  for (long u = static_cast<long>(blockIdx.x) * 256 + threadIdx.x; u < total; u += static_cast<long>(gridDim.x) * 256) {
    const long r = u / chunks;
    const int c = static_cast<int>(u - r * chunks) * 8;
    const T *dh = static_cast<const T *>(a.dh) + r * a.ld_h + c, *gu = static_cast<const T *>(a.gu) + r * a.ld_gu + c;
    T *out = static_cast<T *>(a.dgu) + r * a.ld_dgu + c;
    float d[8], g[8], w[8];
    if (vec) {
      Elem<T>::unpack(ld_stream(dh), d);
      Elem<T>::unpack(ld_stream(gu), g);
      Elem<T>::unpack(ld_stream(gu + a.m), w);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const bool has = c + k < a.m;
        d[k] = has ? Elem<T>::to(dh[k]) : 0.f;
        g[k] = has ? Elem<T>::to(gu[k]) : 0.f;
        w[k] = has ? Elem<T>::to(gu[a.m + k]) : 0.f;
      }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float value, slope;
      act_slope<ACT>(g[k], value, slope);
      g[k] = d[k] * w[k] * slope;
      w[k] = d[k] * value;
    }
    if (vec) {
      *reinterpret_cast<uint4 *>(out) = Elem<T>::pack(g);
      *reinterpret_cast<uint4 *>(out + a.m) = Elem<T>::pack(w);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (c + k < a.m) {
          out[k] = Elem<T>::from(g[k]);
          out[a.m + k] = Elem<T>::from(w[k]);
        }
    }
  }
}

template <typename T>
cudaError_t slope_type(const GatedArgs &a, unsigned grid, bool vec, cudaStream_t s) {
  switch (a.act) {
    case MOE_ACT_SILU: gated_slope_kernel<T, MOE_ACT_SILU><<<grid, 256, 0, s>>>(a, vec); break;
    case MOE_ACT_GELU: gated_slope_kernel<T, MOE_ACT_GELU><<<grid, 256, 0, s>>>(a, vec); break;
    case MOE_ACT_GELU_TANH: gated_slope_kernel<T, MOE_ACT_GELU_TANH><<<grid, 256, 0, s>>>(a, vec); break;
    default: gated_slope_kernel<T, MOE_ACT_RELU><<<grid, 256, 0, s>>>(a, vec); break;
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gated_slope(const GatedArgs &a, int num_sms, cudaStream_t s) {
  if (a.rows == 0) return cudaSuccess;
  HostTrace t("gated_slope", s);
  const auto at16 = [](const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
  const bool vec = at16(a.dh) && at16(a.gu) && at16(a.dgu) && a.ld_h % 8 == 0 && a.ld_gu % 8 == 0 && a.ld_dgu % 8 == 0 &&
                   a.m % 8 == 0;
  const long want = (static_cast<long>(a.rows) * ((a.m + 7) / 8) + 255) / 256, most = num_sms * 16L;
  const unsigned grid = static_cast<unsigned>(want < most ? want : most);
  return a.dtype == MOE_ELEM_BF16 ? slope_type<__nv_bfloat16>(a, grid, vec, s) : slope_type<__half>(a, grid, vec, s);
}

}  // namespace moe
