// gdn2_linattn.h -- argument blocks and launchers of the linear attention with a decay for each head,
// shared between its C entry points and kernels. Not a public header.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "gdn2_internal.h"

namespace gdn2 {

// One sweep of the recurrence Z <- g Z + y_t z_t^T, r_t = Z^T x_t along every (sequence, head): the forward
// (x, y, z) = (q, k, v), and with other roles each gradient (gdn2_linattn.hip). x, y have A channels, z and r have
// E channels; the state is A x E.
struct LinSweep {
  const void* x;
  const void* y;
  const void* z;
  void* r;                       // [rows, H, E] of the inputs' type, or fp32 when r_f32
  int xdiv, ydiv, zdiv;          // head h reads head h / div of the tensor
  bool r_f32;
  bool rev;                      // walk every sequence from its last token to its first
  int first;                     // 1: the entering state is decayed once before the first token, 0: not
  float si, so;                  // scale of y z^T, scale of r
  const float* Z0;               // entering states [N, H, ...], nullable; element (a, e) at a * z0_rs + e * z0_cs
  int z0_rs, z0_cs;
  float* Z1;                     // last states [N, H, A, E], nullable
  float* seg_state;              // [max_segs (x N when dense)][H][A][E]: the state entering each piece
};

constexpr int kLinSweeps = 3;    // sweeps of one launch at most

struct LinArgs {
  LinSweep sw[kLinSweeps];       // of the same A and E, run side by side
  int sweeps;
  const float* log_decay;        // [H]
  int N, T, H, A, E;             // sequences (batch rows), tokens a row (packed: all of them), heads of the states
  bool f32;
  // pieces: the tokens of a sequence are cut into pieces of seg_tok; with more than one, all enter from seg_state
  // (the first too, so that Z1 may be Z0)
  bool pieces;
  int seg_tok;
  int max_segs;                  // dense: pieces of a sequence; packed: bound of all sequences' pieces
  // packed batches: offsets and piece tables on the device (null: dense)
  const int64_t* cu;
  const int* seg_first;
  const int* seg_seq;
};

int linattn_seg_tokens(int N, int T, int H, int E, int sweeps, bool packed, bool f32);
int linattn_max_segs(int N, int T, int seg_tok, bool packed);
// a packed batch's tables, built on the device from the caller's offsets; sets a's pointers to them
size_t linattn_table_bytes(int N, int max_segs);
hipError_t launch_linattn_plan(const int64_t* cu, char* tables, LinArgs& a, hipStream_t s);
// zeros in the rows [row_bytes] of x outside every sequence
hipError_t launch_linattn_outside(void* x, const int64_t* cu, int N, int64_t T, int64_t row_bytes, hipStream_t s);
// piece states of the sweeps, joined and handed to the sweeps' pieces, then the sweeps themselves
hipError_t launch_linattn_sweeps(const LinArgs& a, hipStream_t s);
// dst[row, j, :] = sum over i < G of src[row, j G + i, :] (src fp32), rounded to the type of dst; packed
// batches (cu [N + 1]): for rows cu[0] .. cu[N] - 1 alone
hipError_t launch_linattn_group_sum(const float* src, void* dst, int64_t rows, int heads, int G, int D, bool f32,
                                    const int64_t* cu, int N, hipStream_t s);

struct LinDecodeArgs {
  const void* q;
  const void* k;
  const void* v;
  const float* log_decay;
  float* S;
  void* o;
  const int* slots;              // null: S is [B, H, Dk, Dv]
  int num_slots;
  int B, Hk, H, Dk, Dv;
  float scale;
  bool f32;
};
hipError_t launch_linattn_decode(const LinDecodeArgs& a, hipStream_t s);

}  // namespace gdn2
