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
__global__ void __launch_bounds__(256) gated_slope_kernel(const GatedArgs a) {
  const int chunks = a.m >> 3;
  const long total = static_cast<long>(a.rows) * chunks;
  for (long u = static_cast<long>(blockIdx.x) * 256 + threadIdx.x; u < total; u += static_cast<long>(gridDim.x) * 256) {
    const long r = u / chunks;
    const int c = static_cast<int>(u - r * chunks) * 8;
    const T *dh = static_cast<const T *>(a.dh) + r * a.ld_h + c, *gu = static_cast<const T *>(a.gu) + r * a.ld_gu + c;
    T *out = static_cast<T *>(a.dgu) + r * a.ld_dgu + c;
    float d[8], g[8], w[8];
    Elem<T>::unpack(ld_stream(dh), d);
    Elem<T>::unpack(ld_stream(gu), g);
    Elem<T>::unpack(ld_stream(gu + a.m), w);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float value, slope;
      act_slope<ACT>(g[k], value, slope);
      g[k] = d[k] * w[k] * slope;
      w[k] = d[k] * value;
    }
    *reinterpret_cast<uint4 *>(out) = Elem<T>::pack(g);
    *reinterpret_cast<uint4 *>(out + a.m) = Elem<T>::pack(w);
  }
}

// Rows that are no whole 16-byte pieces: element by element, lanes next to each other.
template <typename T, int ACT>
__global__ void __launch_bounds__(256) gated_slope_any_kernel(const GatedArgs a) {
  const int lane = threadIdx.x & 31, strips = (a.m + 127) >> 7;
  const long total = static_cast<long>(a.rows) * strips;
  for (long u = static_cast<long>(blockIdx.x) * 8 + (threadIdx.x >> 5); u < total; u += static_cast<long>(gridDim.x) * 8) {
    const long r = u / strips;
    const int c0 = static_cast<int>(u - r * strips) * 128 + lane;
    const T *dh = static_cast<const T *>(a.dh) + r * a.ld_h, *gu = static_cast<const T *>(a.gu) + r * a.ld_gu;
    T *out = static_cast<T *>(a.dgu) + r * a.ld_dgu;
    float d[4], g[4], w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = c0 + 32 * k;
      const bool has = c < a.m;
      d[k] = has ? Elem<T>::to(dh[c]) : 0.f;
      g[k] = has ? Elem<T>::to(gu[c]) : 0.f;
      w[k] = has ? Elem<T>::to(gu[a.m + c]) : 0.f;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = c0 + 32 * k;
      float value, slope;
      act_slope<ACT>(g[k], value, slope);
      if (c < a.m) {
        out[c] = Elem<T>::from(d[k] * w[k] * slope);
        out[a.m + c] = Elem<T>::from(d[k] * value);
      }
    }
  }
}

template <typename T, int ACT>
cudaError_t slope_act(const GatedArgs &a, bool vec, int num_sms, cudaStream_t s) {
  const long want = vec ? (static_cast<long>(a.rows) * (a.m >> 3) + 255) / 256 : (static_cast<long>(a.rows) * ((a.m + 127) >> 7) + 7) / 8;
  const long most = num_sms * 16L;
  const unsigned grid = static_cast<unsigned>(want < most ? want : most);
  if (vec) gated_slope_kernel<T, ACT><<<grid, 256, 0, s>>>(a);
  else gated_slope_any_kernel<T, ACT><<<grid, 256, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t slope_type(const GatedArgs &a, bool vec, int num_sms, cudaStream_t s) {
  switch (a.act) {
    case MOE_ACT_SILU: return slope_act<T, MOE_ACT_SILU>(a, vec, num_sms, s);
    case MOE_ACT_GELU: return slope_act<T, MOE_ACT_GELU>(a, vec, num_sms, s);
    case MOE_ACT_GELU_TANH: return slope_act<T, MOE_ACT_GELU_TANH>(a, vec, num_sms, s);
    default: return slope_act<T, MOE_ACT_RELU>(a, vec, num_sms, s);
  }
}

}  // namespace

cudaError_t launch_gated_slope(const GatedArgs &a, int num_sms, cudaStream_t s) {
  if (a.rows == 0) return cudaSuccess;
  HostTrace t("gated_slope", s);
  const auto at16 = [](const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
  const bool vec = at16(a.dh) && at16(a.gu) && at16(a.dgu) && a.ld_h % 8 == 0 && a.ld_gu % 8 == 0 && a.ld_dgu % 8 == 0 &&
                   a.m % 8 == 0;
  return a.dtype == MOE_ELEM_BF16 ? slope_type<__nv_bfloat16>(a, vec, num_sms, s) : slope_type<__half>(a, vec, num_sms, s);
}

}  // namespace moe
