// gdn2_qk_norm.hip -- norms of q and k for each head with the position rotation, in one pass.
//
//   y = R(p) (x r w),  r = (sum x^2 * inv_count + eps)^(-1/2)         inv_count: 1 / D (RMS norm) or 1 (L2 norm)
//   R(p) turns the first `rot` channels in pairs (a, b) by the angle p inv_freq[j]: channels j and j + rot/2, or
//   2j and 2j + 1 (interleaved).
// Backward, with u = R(p)^T dy scale:  dw = sum u x r,  dx = r (h - x r^2 inv_count <h, x>),  h = u w.
//
// HBM-bound: x in, y out (backward: x and dy in, dx out), about 15 operations an element. A wave takes a token, or a
// share of its heads where there are few tokens; D / 8 lanes own a head's row, 8 channels (16 bytes of bf16) a lane.
// 32768 tokens of 16 + 16 heads, D 128, bf16: forward 101 us (5.3 TB/s of 0.54 GB, a copy's rate), backward 181 us: 160
// for the rows (5.0 of 0.81 GB; 215 in all with its rows converted as they arrive) and 21 for the sums of the weights'
// gradients, 16 workgroups that each add 64 values a thread one after another.
// A token's angles are the same for all its heads, so lane j forms the cosine and sine of pair j once (the angle in
// turns in fp64, reduced, then fp32) and the rows read them from LDS.

#include "gdn2_qk_norm.h"

#include "gdn2_common.h"

namespace gdn2 {

namespace {

constexpr int kWaves = 4;        // waves a workgroup
constexpr int kTargetWaves = 4096;  // waves that few tokens are spread over
constexpr int kBwdWorkgroups = 1024;

template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, true));
}
// sum over groups of L neighbouring lanes, in every lane (L = 2, 4, 8, 16)
template <int L>
__device__ __forceinline__ float group_sum(float x) {
  x += dpp<0xB1>(x);                        // lane ^ 1
  if constexpr (L >= 4) x += dpp<0x4E>(x);  // lane ^ 2
  if constexpr (L >= 8) x += dpp<0x141>(x);   // mirrored in 8 lanes
  if constexpr (L >= 16) x += dpp<0x140>(x);  // mirrored in 16 lanes
  return x;
}

template <bool F32>
__device__ __forceinline__ void store8(void* base, int64_t at, const float (&x)[8]) {
  if constexpr (F32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + at);
    p[0] = make_float4(x[0], x[1], x[2], x[3]);
    p[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    bf16x8 b;
#pragma unroll
    for (int e = 0; e < 8; ++e) b[e] = f32_to_bf16(x[e]);
    *reinterpret_cast<bf16x8*>(static_cast<__bf16*>(base) + at) = b;
  }
}

// A token's rotation as a lane with channels 8c..8c+7 applies it: cosines and sines of its channels' pairs.
template <int D, bool PAIRS>
struct Turn {
  float cs[PAIRS ? 4 : 8], sn[PAIRS ? 4 : 8];
  int partner;      // lane with the other channels of the pairs (halves)
  bool on, second;  // the lane's channels turn; they are the pairs' second ones

  __device__ __forceinline__ void setup(int l, int rot) {
    const int c = l & (D / 8 - 1);
    on = 8 * c < rot;
    second = !PAIRS && 16 * c >= rot;
    partner = PAIRS || !on ? l : second ? l - rot / 16 : l + rot / 16;
  }
  // table: [2][64] of this wave
  __device__ __forceinline__ void fetch(float* table, const QkNormArgs& a, int64_t n, int l) {
    const int half = a.rot >> 1;
    const int64_t p0 = n % a.period;
    const int64_t pos = a.pos ? a.pos[p0] : p0;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // the wave's reads of the last token's are before
    if (l < half) {
      double turns = (double)pos * (double)a.inv_freq[l] * 0.15915494309189533577;
      turns -= rint(turns);
      float s, c;
      sincospif(2.f * (float)turns, &s, &c);
      table[l] = c;
      table[64 + l] = s;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    const int c = l & (D / 8 - 1);
    const int j = PAIRS ? 4 * c : 8 * c - (second ? half : 0);
    if (on) {
#pragma unroll
      for (int e = 0; e < (PAIRS ? 4 : 8); ++e) {
        cs[e] = table[j + e];
        sn[e] = table[64 + j + e];
      }
    }
  }
  // x <- R x, or R^T x (BACK); o: the partner lane's channels (halves)
  template <bool BACK>
  __device__ __forceinline__ void turn(float (&x)[8], const float (&o)[8]) const {
    if (!on) return;
    if constexpr (PAIRS) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float u = x[2 * e], v = x[2 * e + 1], s = BACK ? -sn[e] : sn[e];
        x[2 * e] = u * cs[e] - v * s;
        x[2 * e + 1] = v * cs[e] + u * s;
      }
    } else {
      const bool minus = second == BACK;  // the first channels take -sin, the second +sin; R^T the other way
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = x[e] * cs[e] + (minus ? -o[e] : o[e]) * sn[e];
    }
  }
  __device__ __forceinline__ void forward(float (&x)[8]) const {
    float o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = PAIRS ? 0.f : __shfl(x[e], partner);
    turn<false>(x, o);
  }
  // R^T of a row still as it is in memory: its partner's channels travel packed
  template <bool F32>
  __device__ __forceinline__ void back(const Raw8<F32>& r, float (&x)[8]) const {
    cvt(r, x);
    float o[8];
    if constexpr (PAIRS) {
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = 0.f;
    } else if constexpr (F32) {
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = __shfl(x[e], partner);
    } else {
      Raw8<false> p;
      p.u.x = __shfl((int)r.u.x, partner);
      p.u.y = __shfl((int)r.u.y, partner);
      p.u.z = __shfl((int)r.u.z, partner);
      p.u.w = __shfl((int)r.u.w, partner);
      cvt(p, o);
    }
    turn<true>(x, o);
  }
};

// A wave's row steps: q's heads RW at a time, then k's.
template <int D>
struct Steps {
  static constexpr int LPR = D / 8, RW = 64 / LPR;
  int q, all;
  __device__ __host__ __forceinline__ Steps(int Hq, int Hk)
      : q((Hq + RW - 1) / RW), all((Hq + RW - 1) / RW + (Hk + RW - 1) / RW) {}
};

template <int D, bool F32, bool PAIRS>
__global__ __launch_bounds__(64 * kWaves) void gdn2_qk_norm_fwd_kernel(QkNormArgs a, int split) {
  constexpr int LPR = D / 8, RW = 64 / LPR;
  __shared__ float tables[kWaves][128];
  const int l = lane_id(), c = l & (LPR - 1), row = l / LPR;
  const int wv = __builtin_amdgcn_readfirstlane(wave_id());
  const int64_t task = (int64_t)blockIdx.x * kWaves + wv;
  const int64_t n = task / split;
  if (n >= a.tokens) return;
  const int part = (int)(task - n * split);
  const Steps<D> st(a.s[0].heads, a.s[1].heads);
  const int i0 = (int)((int64_t)st.all * part / split), i1 = (int)((int64_t)st.all * (part + 1) / split);
  Turn<D, PAIRS> turn;
  turn.setup(l, a.rot);
  turn.fetch(tables[wv], a, n, l);
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    const QkNormSide& s = a.s[side];
    const int j0 = side == 0 ? i0 : max(i0, st.q) - st.q, j1 = side == 0 ? min(i1, st.q) : i1 - st.q;
    if (j0 >= j1) continue;
    float w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = 1.f;
    if (s.w) load8<true>(s.w, 8 * c, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] *= s.scale;
    constexpr int U = 4;  // rows in flight
    for (int j = j0; j < j1; j += U) {
      float x[U][8];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int head = min(min(j + u, j1 - 1) * RW + row, s.heads - 1);
        load8<F32>(s.x, n * s.x_stride + (int64_t)head * D + 8 * c, x[u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float q = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) q = fmaf(x[u][e], x[u][e], q);
        const float r = 1.f / sqrtf(fmaf(group_sum<LPR>(q), a.inv_count, a.eps));
#pragma unroll
        for (int e = 0; e < 8; ++e) x[u][e] = x[u][e] * r * w[e];
        turn.forward(x[u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int head = (j + u) * RW + row;
        if (j + u < j1 && head < s.heads) store8<F32>(s.y, n * s.y_stride + (int64_t)head * D + 8 * c, x[u]);
      }
    }
  }
}

// Tokens go round the workgroups, so that a wave's sums of the weights' gradients stay in its registers; the
// workgroups' sums are added in a second kernel, in a fixed order.
template <int D, bool F32, bool F32DY, bool PAIRS>
__global__ __launch_bounds__(64 * kWaves, 4) void gdn2_qk_norm_bwd_kernel(QkNormArgs a, int split) {
  constexpr int LPR = D / 8, RW = 64 / LPR;
  __shared__ float tables[kWaves][128];
  __shared__ float sums[kWaves][2][D];
  const int l = lane_id(), c = l & (LPR - 1), row = l / LPR;
  const int wv = __builtin_amdgcn_readfirstlane(wave_id());
  const Steps<D> st(a.s[0].heads, a.s[1].heads);
  Turn<D, PAIRS> turn;
  turn.setup(l, a.rot);
  float dw[2][8], w[2][8];
#pragma unroll
  for (int side = 0; side < 2; ++side) {
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[side][e] = 0.f, w[side][e] = 1.f;
    if (a.s[side].w) load8<true>(a.s[side].w, 8 * c, w[side]);
  }
  const int64_t tasks = a.tokens * split;
  for (int64_t task = (int64_t)blockIdx.x * kWaves + wv; task < tasks; task += (int64_t)gridDim.x * kWaves) {
    const int64_t n = task / split;
    const int part = (int)(task - n * split);
    const int i0 = (int)((int64_t)st.all * part / split), i1 = (int)((int64_t)st.all * (part + 1) / split);
    turn.fetch(tables[wv], a, n, l);
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const QkNormSide& s = a.s[side];
      const int j0 = side == 0 ? i0 : max(i0, st.q) - st.q, j1 = side == 0 ? min(i1, st.q) : i1 - st.q;
      constexpr int U = F32 || F32DY ? 2 : 4;  // rows in flight, as they are in memory
      for (int j = j0; j < j1; j += U) {
        Raw8<F32> xr[U];
        Raw8<F32DY> dr[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int head = min(min(j + u, j1 - 1) * RW + row, s.heads - 1);
          ld_raw(xr[u], s.x, n * s.x_stride + (int64_t)head * D + 8 * c);
          ld_raw(dr[u], s.dy, (n * s.heads + head) * D + 8 * c);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (j + u >= j1) break;
          const int head = (j + u) * RW + row;
          const bool ok = head < s.heads;
          float x[8], d[8];
          turn.back(dr[u], d);
          cvt(xr[u], x);
          float q = 0.f, p = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            d[e] *= s.scale;
            q = fmaf(x[e], x[e], q);
            p = fmaf(x[e], d[e] * w[side][e], p);
          }
          const float r = 1.f / sqrtf(fmaf(group_sum<LPR>(q), a.inv_count, a.eps));
          const float t = group_sum<LPR>(p) * a.inv_count * r * r;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (ok) dw[side][e] = fmaf(d[e] * x[e], r, dw[side][e]);
            x[e] = r * (d[e] * w[side][e] - x[e] * t);
          }
          if (ok) store8<F32>(s.y, n * s.y_stride + (int64_t)head * D + 8 * c, x);
        }
      }
    }
  }
  if (a.partial == nullptr) return;
#pragma unroll
  for (int side = 0; side < 2; ++side)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float v = dw[side][e];
#pragma unroll
      for (int off = LPR; off < 64; off *= 2) v += __shfl_xor(v, off);
      if (row == 0) sums[wv][side][8 * c + e] = v;
    }
  __syncthreads();
  for (int j = threadIdx.x; j < 2 * D; j += 64 * kWaves) {
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < kWaves; ++k) v += (&sums[k][0][0])[j];
    a.partial[(int64_t)blockIdx.x * 2 * D + j] = v;
  }
}

// 16 columns of the partial sums a workgroup, 16 threads a column.
__global__ __launch_bounds__(256) void gdn2_qk_norm_dw_kernel(QkNormArgs a, int rows) {
  __shared__ float red[16][17];
  const int c = threadIdx.x & 15, r = threadIdx.x >> 4, col = blockIdx.x * 16 + c;
  float v = 0.f;
  for (int j = r; j < rows; j += 16) v += a.partial[(int64_t)j * 2 * a.D + col];
  red[r][c] = v;
  __syncthreads();
  if (r == 0) {
    v = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) v += red[j][c];
    const int side = col >= a.D;
    if (a.s[side].dw) a.s[side].dw[col - side * a.D] = v;
  }
}

int steps_of(int Hq, int Hk, int D) {
  const int rw = 512 / D;
  return (Hq + rw - 1) / rw + (Hk + rw - 1) / rw;
}

// waves a token
int split_of(int64_t tokens, int steps) {
  int64_t s = (kTargetWaves + tokens - 1) / tokens;
  if (s > steps) s = steps;
  return s < 1 ? 1 : (int)s;
}

template <int D, bool F32, bool PAIRS>
hipError_t fwd_t(const QkNormArgs& a, hipStream_t s) {
  const int split = split_of(a.tokens, steps_of(a.s[0].heads, a.s[1].heads, D));
  const int64_t blocks = (a.tokens * split + kWaves - 1) / kWaves;
  hipLaunchKernelGGL((gdn2_qk_norm_fwd_kernel<D, F32, PAIRS>), dim3((unsigned)blocks), dim3(64 * kWaves), 0, s, a,
                     split);
  return hipGetLastError();
}

template <int D, bool F32, bool F32DY, bool PAIRS>
hipError_t bwd_t(const QkNormArgs& a, hipStream_t s) {
  const int split = split_of(a.tokens, steps_of(a.s[0].heads, a.s[1].heads, D));
  const int blocks = qk_norm_bwd_workgroups(a.tokens, a.s[0].heads, a.s[1].heads, D);
  hipLaunchKernelGGL((gdn2_qk_norm_bwd_kernel<D, F32, F32DY, PAIRS>), dim3((unsigned)blocks), dim3(64 * kWaves), 0, s,
                     a, split);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.partial == nullptr) return e;
  hipLaunchKernelGGL(gdn2_qk_norm_dw_kernel, dim3(2 * D / 16), dim3(256), 0, s, a, blocks);
  return hipGetLastError();
}

template <int D>
hipError_t fwd_d(const QkNormArgs& a, hipStream_t s) {
  if (a.f32) return a.interleaved ? fwd_t<D, true, true>(a, s) : fwd_t<D, true, false>(a, s);
  return a.interleaved ? fwd_t<D, false, true>(a, s) : fwd_t<D, false, false>(a, s);
}

template <int D>
hipError_t bwd_d(const QkNormArgs& a, hipStream_t s) {
  if (a.f32) return a.interleaved ? bwd_t<D, true, true, true>(a, s) : bwd_t<D, true, true, false>(a, s);
  if (a.f32_dy) return a.interleaved ? bwd_t<D, false, true, true>(a, s) : bwd_t<D, false, true, false>(a, s);
  return a.interleaved ? bwd_t<D, false, false, true>(a, s) : bwd_t<D, false, false, false>(a, s);
}

}  // namespace

int qk_norm_bwd_workgroups(int64_t tokens, int Hq, int Hk, int D) {
  const int64_t blocks = (tokens * split_of(tokens, steps_of(Hq, Hk, D)) + kWaves - 1) / kWaves;
  return (int)(blocks < kBwdWorkgroups ? blocks : kBwdWorkgroups);
}

hipError_t launch_qk_norm_fwd(const QkNormArgs& a, hipStream_t s) {
  switch (a.D) {
    case 16: return fwd_d<16>(a, s);
    case 32: return fwd_d<32>(a, s);
    case 64: return fwd_d<64>(a, s);
    case 128: return fwd_d<128>(a, s);
  }
  return hipErrorInvalidValue;
}

hipError_t launch_qk_norm_bwd(const QkNormArgs& a, hipStream_t s) {
  switch (a.D) {
    case 16: return bwd_d<16>(a, s);
    case 32: return bwd_d<32>(a, s);
    case 64: return bwd_d<64>(a, s);
    case 128: return bwd_d<128>(a, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace gdn2
