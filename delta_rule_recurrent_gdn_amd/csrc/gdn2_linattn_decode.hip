// gdn2_linattn_decode.hip -- one token of the linear attention with a decay for each head.
//
// Per (entry, head), state S [Dk, Dv] fp32 in place:  S <- g S + k v^T,  o = scale S^T q.
//
// HBM-bound: 8 Dk Dv bytes of state an entry and head, five operations an element. One workgroup per (entry, head);
// a thread owns 4 neighbouring value columns of RPT key rows, so every access of a wave is one contiguous block.
// 256 entries of 16 heads, d 128 (0.54 GB): 109 us, 4.9 TB/s, with the states out of the caches; one entry: 4 us.
// The new state goes out as soon as it is formed; only the column sums of o meet in LDS. It goes through plain
// pointers: a 16-byte buffer store with a scalar offset, followed at once by a vector instruction that overwrites its
// data register, stored the new value in some lanes (no wait is put between the two for that form of store).

#include "gdn2_common.h"
#include "gdn2_linattn.h"

namespace gdn2 {

template <int DK, int DV>
struct LinDecodeShape {
  static constexpr int kCols4 = DV / 4;
  static constexpr int kThreads = (kCols4 * DK < 256) ? kCols4 * DK : 256;
  static constexpr int kGroups = kThreads / kCols4;  // key rows side by side
  static constexpr int kRows = DK / kGroups;         // key rows a thread
  static_assert(kRows >= 1 && kGroups * kRows == DK, "decode tiling");
};

template <int DK, int DV, bool F32>
__global__ __launch_bounds__((LinDecodeShape<DK, DV>::kThreads)) void gdn2_linattn_decode_kernel(LinDecodeArgs a) {
  using Sh = LinDecodeShape<DK, DV>;
  constexpr int NT = Sh::kThreads, RG = Sh::kGroups, RPT = Sh::kRows, C4 = Sh::kCols4;
  __shared__ float red[RG][DV + 4];
  const int tid = threadIdx.x;
  const int64_t bh = blockIdx.x;
  const int b = (int)(bh / a.H), h = (int)(bh - (int64_t)b * a.H);
  int64_t state = bh;
  if (a.slots) {
    const int slot = a.slots[b];
    if (slot < 0 || slot >= a.num_slots) {  // no state: o = 0, nothing else
      for (int j = tid; j < DV; j += NT) {
        if constexpr (F32) static_cast<float*>(a.o)[bh * DV + j] = 0.f;
        else static_cast<uint16_t*>(a.o)[bh * DV + j] = 0;
      }
      return;
    }
    state = (int64_t)slot * a.H + h;
  }
  const int j4 = tid % C4, rg = tid / C4;
  float4* const S = reinterpret_cast<float4*>(a.S + state * (int64_t)(DK * DV)) + tid;
  constexpr int kStep = RG * C4;
  float4 s[RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i)
    s[i] = S[i * kStep];
  const int64_t qk = ((int64_t)b * a.Hk + h / (a.H / a.Hk)) * DK;
  float v[4], q[RPT], k[RPT];
  load4<F32>(a.v, bh * DV + 4 * j4, v);
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    q[i] = load1<F32>(a.q, qk + rg + RG * i);
    k[i] = load1<F32>(a.k, qk + rg + RG * i);
  }
  // the decay and what rounding left of it: a state is multiplied by it at every token, always off to the same side
  const double decay = exp((double)a.log_decay[h]);
  const float g = (float)decay, rest = g <= 3.4028235e38f ? (float)(decay - g) : 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    s[i].x = fmaf(g, s[i].x, fmaf(rest, s[i].x, k[i] * v[0]));
    s[i].y = fmaf(g, s[i].y, fmaf(rest, s[i].y, k[i] * v[1]));
    s[i].z = fmaf(g, s[i].z, fmaf(rest, s[i].z, k[i] * v[2]));
    s[i].w = fmaf(g, s[i].w, fmaf(rest, s[i].w, k[i] * v[3]));
    o.x = fmaf(q[i], s[i].x, o.x); o.y = fmaf(q[i], s[i].y, o.y);
    o.z = fmaf(q[i], s[i].z, o.z); o.w = fmaf(q[i], s[i].w, o.w);
    S[i * kStep] = s[i];
  }
  *reinterpret_cast<float4*>(&red[rg][4 * j4]) = o;
  __syncthreads();
  for (int j = tid; j < DV; j += NT) {
    float x = 0.f;
#pragma unroll
    for (int r = 0; r < RG; ++r) x += red[r][j];
    x *= a.scale;
    if constexpr (F32) static_cast<float*>(a.o)[bh * DV + j] = x;
    else static_cast<__bf16*>(a.o)[bh * DV + j] = f32_to_bf16(x);
  }
}

template <int DK, int DV, bool F32>
static hipError_t launch_lin_decode_t(const LinDecodeArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((gdn2_linattn_decode_kernel<DK, DV, F32>), dim3((unsigned)((int64_t)a.B * a.H)),
                     dim3(LinDecodeShape<DK, DV>::kThreads), 0, s, a);
  return hipGetLastError();
}

template <int DK, bool F32>
static hipError_t launch_lin_decode_dv(const LinDecodeArgs& a, hipStream_t s) {
  switch (a.Dv) {
    case 16: return launch_lin_decode_t<DK, 16, F32>(a, s);
    case 32: return launch_lin_decode_t<DK, 32, F32>(a, s);
    case 64: return launch_lin_decode_t<DK, 64, F32>(a, s);
    case 128: return launch_lin_decode_t<DK, 128, F32>(a, s);
  }
  return hipErrorInvalidValue;
}

template <bool F32>
static hipError_t launch_lin_decode_dk(const LinDecodeArgs& a, hipStream_t s) {
  switch (a.Dk) {
    case 16: return launch_lin_decode_dv<16, F32>(a, s);
    case 32: return launch_lin_decode_dv<32, F32>(a, s);
    case 64: return launch_lin_decode_dv<64, F32>(a, s);
    case 128: return launch_lin_decode_dv<128, F32>(a, s);
  }
  return hipErrorInvalidValue;
}

hipError_t launch_linattn_decode(const LinDecodeArgs& a, hipStream_t s) {
  return a.f32 ? launch_lin_decode_dk<true>(a, s) : launch_lin_decode_dk<false>(a, s);
}

}  // namespace gdn2
