// gdn2_linattn.hip -- linear attention with a decay for each head: launchers of the sweeps, the join of the piece
// states, the sum over shared heads.
//
// A sequence of few (sequence, head) pairs leaves most of the GPU idle when one workgroup walks it whole, so it is cut
// into pieces: a first pass sums every piece's own contribution to the state (it reads y and z alone), the join kernel
// runs Z_in[s+1] = g^L Z_in[s] + U[s] over the pieces of a sequence, element by element, and the sweep then walks all
// pieces at once. The price is a second read of y and z.

#include "gdn2_linattn.h"

#include "gdn2_common.h"

namespace gdn2 {

// by operand type, one translation unit each
hipError_t launch_linattn_bf16(const LinArgs& a, bool state, hipStream_t s);
hipError_t launch_linattn_f32(const LinArgs& a, bool state, hipStream_t s);

namespace {

constexpr int kJoinThreads = 256;

// One thread an element quadruple of a (sequence, head)'s state: the pieces one after another, the next one's sum sent
// for ahead. Latency-bound: 6 us for the 8 pieces of 16 heads of d 128 (17 MB, from the caches).
__global__ __launch_bounds__(kJoinThreads) void gdn2_linattn_join_kernel(LinArgs a, int blocks) {
  const LinSweep& sw = a.sw[blockIdx.y];
  const int chain = blockIdx.x / blocks;
  const int n = chain / a.H, h = chain - n * a.H;
  const int at = ((blockIdx.x % blocks) * kJoinThreads + threadIdx.x) * 4;
  if (at >= a.A * a.E) return;
  const int row = at / a.E, col = at % a.E;
  int nseg, slot, step;
  if (a.cu) {
    slot = a.seg_first[n];
    nseg = a.seg_first[n + 1] - slot;
    step = 1;
  } else {
    slot = n;
    nseg = a.max_segs;
    step = a.N;
  }
  const int64_t state = (int64_t)a.A * a.E;
  float z[4] = {0.f, 0.f, 0.f, 0.f};
  if (sw.Z0) {
    const float* src = sw.Z0 + (int64_t)chain * state;
#pragma unroll
    for (int e = 0; e < 4; ++e) z[e] = src[(int64_t)row * sw.z0_rs + (int64_t)(col + e) * sw.z0_cs];
  }
  if (nseg == 0) {  // a sequence without tokens: its last state is its first
    if (sw.Z1) *reinterpret_cast<float4*>(sw.Z1 + (int64_t)chain * state + at) = make_float4(z[0], z[1], z[2], z[3]);
    return;
  }
  if (!a.pieces) return;
  const float ld = a.log_decay[h];
  const double d = exp((ld < -1e4f ? -1e4 : (double)ld) * a.seg_tok);
  const float hi = (float)d, lo = hi <= 3.4028235e38f ? (float)(d - hi) : 0.f;
  float4* p = reinterpret_cast<float4*>(sw.seg_state + ((int64_t)slot * a.H + h) * state + at);
  const int64_t stride = (int64_t)step * a.H * state / 4;
  p[0] = make_float4(z[0], z[1], z[2], z[3]);
  float4 next = nseg > 1 ? p[stride] : make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s = 1; s < nseg; ++s) {
    const float4 u = next;
    if (s + 1 < nseg) next = p[(s + 1) * stride];
    const float add[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e)  // a state of zeros stays as it is, also where growth over a piece is no fp32 number
      z[e] = z[e] == 0.f ? add[e] : fmaf(z[e], hi, fmaf(z[e], lo, add[e]));
    p[s * stride] = make_float4(z[0], z[1], z[2], z[3]);
  }
}

// Tables of a packed batch, by one wave: cu' (the offsets made non-decreasing within [0, T]), the first piece of every
// sequence, the sequence of every piece (-1 past the last, up to max_segs). 64 sequences at a time, by wave scans: a
// batch of 11 takes 3 us, the delta rule's planner, which scans 1024 offsets in a workgroup, 7.
__global__ __launch_bounds__(64) void gdn2_linattn_plan_kernel(const int64_t* cu_in, int N, int T, int seg_tok,
                                                               int max_segs, int64_t* cu, int* seg_first,
                                                               int* seg_seq) {
  const int l = threadIdx.x;
  int64_t top = 0;   // the largest offset so far
  int first = 0;     // pieces so far
  for (int n0 = 0; n0 <= N; n0 += 64) {
    const int n = n0 + l;
    // offsets n0 .. n0 + 63 and the one after them, as running maxima
    int64_t c = n <= N ? cu_in[n] : 0;
    c = c < 0 ? 0 : c > T ? T : c;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int64_t o = __shfl_up(c, d);
      if (l >= d && o > c) c = o;
    }
    if (c < top) c = top;
    int64_t next = n0 + 64 <= N ? cu_in[n0 + 64] : 0;
    next = next < 0 ? 0 : next > T ? T : next;
    const int64_t last = __shfl(c, 63);
    if (next < last) next = last;
    const int64_t o = __shfl_down(c, 1);
    const int64_t end = l < 63 ? o : next;
    const int own = n < N ? (int)((end - c + seg_tok - 1) / seg_tok) : 0;
    int sum = own;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int o2 = __shfl_up(sum, d);
      if (l >= d) sum += o2;
    }
    const int mine = first + sum - own;
    if (n <= N) {
      cu[n] = c;
      seg_first[n] = mine;
    }
    for (int s = 0; s < own; ++s) seg_seq[mine + s] = n;
    first += __shfl(sum, 63);
    top = last;
  }
  for (int s = first + l; s < max_segs; s += 64) seg_seq[s] = -1;
}

// Zeros in the rows outside every sequence of a packed batch: what the offsets leave, 3 us where that is nothing
// (clearing the whole output first costs its bytes once more).
__global__ __launch_bounds__(256) void gdn2_linattn_outside_kernel(uint4* x, const int64_t* cu, int N, int64_t T,
                                                                   int64_t row16) {
  int64_t lo = 0, hi = 0;  // rows [0, lo) and [hi, T) are outside: the first offset, the largest one
  for (int n = threadIdx.x; n <= N; n += 256) {
    const int64_t c = cu[n] < 0 ? 0 : cu[n] > T ? T : cu[n];
    if (c > hi) hi = c;
  }
  lo = cu[0] < 0 ? 0 : cu[0] > T ? T : cu[0];
  __shared__ int64_t top[256];
  top[threadIdx.x] = hi;
  __syncthreads();
  for (int d = 128; d > 0; d /= 2) {
    if ((int)threadIdx.x < d && top[threadIdx.x + d] > top[threadIdx.x]) top[threadIdx.x] = top[threadIdx.x + d];
    __syncthreads();
  }
  hi = top[0] < lo ? lo : top[0];
  const int64_t n16 = (lo + T - hi) * row16;
  for (int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x; k < n16; k += (int64_t)gridDim.x * 256)
    x[k < lo * row16 ? k : k - lo * row16 + hi * row16] = make_uint4(0u, 0u, 0u, 0u);
}

// dq, dk of shared heads: the sum over the G heads of a group, in their order (no atomics, the same bits every time).
// HBM-bound for long inputs; 2 x 2055 tokens of 4 groups: 4 us, the price of the launch.
template <bool F32>
__global__ __launch_bounds__(256) void gdn2_linattn_group_sum_kernel(const float* src, void* dst, int64_t n4, int heads,
                                                                      int G, int D, const int64_t* cu, int N) {
  // packed: the rows of the sequences alone
  const int64_t row_size = (int64_t)heads * D;
  const int64_t lo = cu ? cu[0] * row_size : 0, hi = cu ? cu[N] * row_size : n4 * 4;
  for (int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x; id < n4; id += (int64_t)gridDim.x * 256) {
    const int64_t at = id * 4;                      // element of [rows, heads, D]
    if (at < lo || at >= hi) continue;
    const int64_t rh = at / D;
    const int d = (int)(at - rh * D);
    const float* p = src + rh * G * D + d;
    float4 s = *reinterpret_cast<const float4*>(p);
    for (int i = 1; i < G; ++i) {
      const float4 x = *reinterpret_cast<const float4*>(p + (int64_t)i * D);
      s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
    }
    if constexpr (F32) st4(static_cast<float*>(dst) + at, s.x, s.y, s.z, s.w);
    else st4(static_cast<__bf16*>(dst) + at, s.x, s.y, s.z, s.w);
  }
}

}  // namespace

// Tokens a piece: about as many pieces as give every CU its one workgroup (the sweeps' LDS holds one; twice as many, in
// two rounds: 64K tokens of 16 heads, forward, 443 -> 465 us, 2 x 2055 tokens, backward, 79 -> 102), of at least four
// chunks (fewer cost more in states written, joined and read than the shorter walk saves: 2 x 2055 tokens of 12
// heads, backward, 115 us with four chunks a piece, 137 with two, 118 with eight; fp32, 2 x 1001 of 8 heads, whose
// chunks are half as long: 27 us with four, 36 with eight, 56 with sixteen). It is no exact round: past 128 heads and
// column groups of all sequences there is one piece each; a backward of equal head sizes is counted with two sweeps
// and runs three; a packed batch is cut as one row of tokens, and every sequence's last piece comes on top (11 prompts
// of 14029 tokens: 336 to 368 workgroups by their lengths).
int linattn_seg_tokens(int N, int T, int H, int E, int sweeps, bool packed, bool f32) {
  constexpr int kUnit = 64, kWorkgroups = 256;
  const int64_t units = (T + kUnit - 1) / kUnit, least = f32 ? 2 : 4;
  const int64_t wide = (int64_t)H * ((E + 63) / 64) * sweeps;  // workgroups a piece
  int64_t L;
  if (packed) {
    L = (units * wide + kWorkgroups - 1) / kWorkgroups;
  } else {
    const int64_t pieces = N * wide >= kWorkgroups ? 1 : kWorkgroups / (N * wide);  // one round of workgroups
    L = (units + pieces - 1) / pieces;
  }
  if (L < least) L = least;
  if (L > units) L = units;
  return (int)(L * kUnit);
}

int linattn_max_segs(int N, int T, int seg_tok, bool packed) {
  return packed ? T / seg_tok + N : (T + seg_tok - 1) / seg_tok;
}

size_t linattn_table_bytes(int N, int max_segs) {
  const auto al = [](size_t x) { return (x + 255) & ~(size_t)255; };
  return al((size_t)(N + 1) * 8) + al((size_t)(N + 1) * 4) + al((size_t)max_segs * 4);
}

hipError_t launch_linattn_plan(const int64_t* cu, char* tables, LinArgs& a, hipStream_t s) {
  const auto al = [](size_t x) { return (x + 255) & ~(size_t)255; };
  int64_t* const out = reinterpret_cast<int64_t*>(tables);
  int* const first = reinterpret_cast<int*>(tables + al((size_t)(a.N + 1) * 8));
  int* const seq = reinterpret_cast<int*>(tables + al((size_t)(a.N + 1) * 8) + al((size_t)(a.N + 1) * 4));
  a.cu = out;
  a.seg_first = first;
  a.seg_seq = seq;
  hipLaunchKernelGGL(gdn2_linattn_plan_kernel, dim3(1), dim3(64), 0, s, cu, a.N, a.T, a.seg_tok, a.max_segs, out, first,
                     seq);
  return hipGetLastError();
}

hipError_t launch_linattn_outside(void* x, const int64_t* cu, int N, int64_t T, int64_t row_bytes, hipStream_t s) {
  hipLaunchKernelGGL(gdn2_linattn_outside_kernel, dim3(512), dim3(256), 0, s, static_cast<uint4*>(x), cu, N, T,
                     row_bytes / 16);
  return hipGetLastError();
}

hipError_t launch_linattn_sweeps(const LinArgs& a, hipStream_t s) {
  const auto run = a.f32 ? launch_linattn_f32 : launch_linattn_bf16;
  if (a.pieces) {
    const hipError_t e = run(a, true, s);
    if (e != hipSuccess) return e;
  }
  bool last = false;
  for (int i = 0; i < a.sweeps; ++i) last |= a.sw[i].Z1 != nullptr;
  if (a.pieces || (a.cu && last)) {
    const int blocks = (a.A * a.E / 4 + kJoinThreads - 1) / kJoinThreads;
    hipLaunchKernelGGL(gdn2_linattn_join_kernel, dim3((unsigned)(a.N * a.H * blocks), a.sweeps), dim3(kJoinThreads), 0,
                       s, a, blocks);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return run(a, false, s);
}

hipError_t launch_linattn_group_sum(const float* src, void* dst, int64_t rows, int heads, int G, int D, bool f32,
                                    const int64_t* cu, int N, hipStream_t s) {
  const int64_t n4 = rows * heads * D / 4;
  if (n4 == 0) return hipSuccess;
  int64_t blocks = (n4 + 255) / 256;
  if (blocks > 8192) blocks = 8192;
  if (f32)
    hipLaunchKernelGGL((gdn2_linattn_group_sum_kernel<true>), dim3((unsigned)blocks), dim3(256), 0, s, src, dst, n4,
                       heads, G, D, cu, N);
  else
    hipLaunchKernelGGL((gdn2_linattn_group_sum_kernel<false>), dim3((unsigned)blocks), dim3(256), 0, s, src, dst, n4,
                       heads, G, D, cu, N);
  return hipGetLastError();
}

}  // namespace gdn2
