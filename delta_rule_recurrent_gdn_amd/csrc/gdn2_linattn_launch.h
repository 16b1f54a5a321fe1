// gdn2_linattn_launch.h -- dispatch of a sweep's sizes to its kernel.
#pragma once

#include "gdn2_linattn_impl.h"

namespace gdn2 {

template <int A, int NW, bool F32, bool STATE>
static hipError_t launch_lin_t(const LinArgs& a, hipStream_t s) {
  using Sh = LinShape<A, NW, F32>;
  constexpr int lds = STATE ? Sh::kLdsState : Sh::kLds;
  const auto kernel = gdn2_linattn_kernel<A, NW, F32, STATE>;
  if (lds > 64 * 1024) {  // more than a launch takes without asking
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  const int64_t items = (int64_t)a.max_segs * (a.cu ? 1 : a.N) * a.H;
  const int64_t blocks = (items + 7) / 8 * 8 * ((a.E + Sh::CW - 1) / Sh::CW) * a.sweeps;
  hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(Sh::kThreads), lds, s, a);
  return hipGetLastError();
}

template <int A, bool F32, bool STATE>
static hipError_t launch_lin_e(const LinArgs& a, hipStream_t s) {
  switch (a.E) {
    case 16: return launch_lin_t<A, 1, F32, STATE>(a, s);
    case 32: return launch_lin_t<A, 2, F32, STATE>(a, s);
    case 64:
    case 128: return launch_lin_t<A, 4, F32, STATE>(a, s);
  }
  return hipErrorInvalidValue;
}

template <bool F32>
static hipError_t launch_lin_a(const LinArgs& a, bool state, hipStream_t s) {
  switch (a.A) {
    case 16: return state ? launch_lin_e<16, F32, true>(a, s) : launch_lin_e<16, F32, false>(a, s);
    case 32: return state ? launch_lin_e<32, F32, true>(a, s) : launch_lin_e<32, F32, false>(a, s);
    case 64: return state ? launch_lin_e<64, F32, true>(a, s) : launch_lin_e<64, F32, false>(a, s);
    case 128: return state ? launch_lin_e<128, F32, true>(a, s) : launch_lin_e<128, F32, false>(a, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace gdn2
