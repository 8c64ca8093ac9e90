// Host-side launchers and argument blocks of the token mixers (internal to the library): linear attention with a decay
// for each head, attention with a sliding window and first tokens that stay visible.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kda_mixers.h"
#include "layer_launch.h"

namespace kda {

// ---- linear attention

// Which state of an array: none (zeros), one a sequence, one a segment, or, of an array with one at the start of each segment and
// one at the end of each sequence, that at the segment's start or the one behind it.
enum { kStateNone = 0, kStateSeq = 1, kStateSeg = 2, kStateStart = 3, kStateEnd = 4 };

// Tokens of a chunk. Twice as many halve what is done once a chunk (the state's scaling and splitting, barriers), but each wave then
// holds twice the rows of outputs and of the next chunk: 157, 159 us for the two walks without dot, where 32 took 140, 133 us
// (B=4, T=4096, HV=32; 120, 116 now), and their tiles with w's leave room for one workgroup a CU.
constexpr int kLinChunk = 32;

// What a walk over the chunks of a segment computes. Rows x, y [tokens, P] and z [tokens, R] of a head; state [P, R]:
//   out_i = in_i (x_i state) + sum_j pair_ij (x_i.y_j) z_j,   state <- decay state + sum_j up_j y_j z_j^T
// over j <= i going forward in time, j >= i going backward.
struct LinArgs {
  Seqs sq;
  int seg;                    // tokens of a segment, a multiple of a chunk's
  int64_t nseg;
  int HV, rep;                // value heads, value heads that share a q/k head
  int P, R;
  int tile;                   // columns of a workgroup: 64 or 128
  int x_qk, y_qk, z_qk;       // rows belong to q/k heads
  const void *x, *y, *z;
  int64_t x_row, y_row, z_row;
  int vec;                    // rows of x, y, z, w and out allow loads of 16 bytes
  const float* g;
  int g_const;
  float scale;
  const float* s0;            // state at the start: kState*
  int s0_mode;
  float *fin, *fin2;          // state at the end
  int fin_mode, fin2_mode;
  float* copy0;               // the state at the start again (entry segment + sequence)
  int64_t s_p, s_r;           // elements between two rows and two columns of a state
  int svec;                   // s_p is 1 and states allow loads of four rows
  float* seg_decay;           // [nseg][HV] decay over a segment, or nullptr
  void* out;                  // [tokens][HV][R] of the type, or fp32 where out_f32
  int out_f32;
  const void* w;              // rows [tokens, R] whose products with out are wanted
  int64_t w_row;
  int w_qk;
  float* dot;                 // [tiles][HV][tokens]
};
// kLinState: only the state. kLinOut, kLinOutRev: out is rounded to the type. kLinDot, kLinDotRev: out, and to fp32's precision what the
// decays' gradients need of it.
enum { kLinState = 0, kLinStateRev, kLinOut, kLinOutFin, kLinOutRev, kLinDot, kLinDotRev };
struct LinCut {
  int seg, tile_k, tile_v;    // tokens of a segment, columns of a tile of K and of V
};
LinCut lin_cut(int dtype, int64_t longest, int64_t heads, int K, int V);
hipError_t launch_lin_walk(int dtype, int mode, const LinArgs& a, hipStream_t st);
template <bool VEC>
hipError_t lin_walk_f32(int mode, const LinArgs& a, hipStream_t st);
template <bool VEC>
hipError_t lin_walk_bf16(int mode, const LinArgs& a, hipStream_t st);
template <bool VEC>
hipError_t lin_walk_dot_bf16(int mode, const LinArgs& a, hipStream_t st);

struct LinScanArgs {
  Seqs sq;
  int seg;
  int64_t nseg;
  int HV;
  int64_t KV;                 // elements of a state
  int slice;                  // of them a workgroup carries
  const float* seg_decay;     // [nseg][HV]
  const float* first;         // [N] states to begin with, or nullptr
  float* states;              // forward: entries segment + sequence; backward: [nseg]
  float* last;                // [N] states at the end, or nullptr
  const float* fwd;           // backward: the forward's states, for dot; or nullptr
  float* dot;                 // [slices][nseg][HV] products of a state's gradient with the state, per slice
  int local;                  // states hold what the segments add
};
// Elements of a state that a workgroup of the scan carries, from the most segments that a sequence has. Many segments are a chain
// of loads, cut into more and longer batches; few are a copy (us of the reverse and the forward scan: four segments of B=4,
// HV=32, 1024 elements 19, 14, 256 elements 40, 27; 25 segments of 4 heads in fp32 14, 12 and 9, 8).
int lin_scan_slice(int64_t segments);
int64_t lin_scan_slices(int64_t KV, int slice);
hipError_t launch_lin_scan(const LinScanArgs& a, bool rev, hipStream_t st);

struct LinGateArgs {
  Seqs sq;
  int seg;
  int64_t nseg;
  int HV, qtiles, ktiles;
  int64_t slices;             // 0: no state behind the segments
  const float *dotq, *dotk, *dots;
  float* dg;                  // [tokens][HV] or, with part, [HV]
  double* part;               // [nseg][HV], or nullptr
};
hipError_t launch_lin_gate(const LinGateArgs& a, hipStream_t st);

// out [tokens][H][W] = sum over the rep heads of a group of in [tokens][H rep][W]
hipError_t launch_group_sum(int dtype, const float* in, void* out, int64_t rows, int rep, int W, hipStream_t st);

struct LinStepArgs {
  int B, H, HV, K, V, slots_n, g_const;
  float scale;
  int64_t q_row, k_row, v_row;
  const void *q, *k, *v;
  const float* g;
  const int32_t* slots;
  float* state;
  void* o;
};
hipError_t launch_lin_step(int dtype, const LinStepArgs& a, hipStream_t st);

// ---- window attention

struct WinArgs {
  Seqs sq;
  int H, HK, D, window, sinks;
  float scale;
  int64_t q_row, k_row, v_row;
  const void *q, *k, *v;
  int vec;                    // rows of all tensors allow loads of 16 bytes
  void* o;
  float* lse;                 // [tokens][H], natural logarithm; or nullptr
  int64_t blocks;             // runs of queries (or keys) over all sequences
  // backward
  const void *out, *dout;
  const float* lse_in;
  float* delta;               // [tokens][H]: do.o of each row, from the gradient of the queries for that of the keys
  void *dq, *dk, *dv;
  int part_len;               // queries of a part behind the window
  int64_t parts;              // parts over all sequences
  float* part;                // [parts + N][sinks][HK][2][D]: the parts, then what the window gives
};
struct WinPlan {
  int qrows, krows;           // queries of a forward block, keys of a backward block
};
WinPlan win_plan(int dtype, int D, int64_t total, int N, int H, int HK);
hipError_t launch_win_fwd(int dtype, const WinArgs& a, int qrows, hipStream_t st);
hipError_t launch_win_cache(int dtype, const WinArgs& a, void* k_cache, void* v_cache, hipStream_t st);
hipError_t launch_win_dq(int dtype, const WinArgs& a, int qrows, hipStream_t st);
hipError_t launch_win_dkv(int dtype, const WinArgs& a, int krows, hipStream_t st);
hipError_t launch_win_sinks(int dtype, const WinArgs& a, hipStream_t st);

struct WinStepArgs {
  int B, H, HK, D, window, sinks, slots_n;
  float scale;
  int64_t q_row, k_row, v_row;
  const void *q, *k, *v;
  const int32_t *pos, *slots;
  void *k_cache, *v_cache, *o;
  int vec;                    // rows of q and of the caches allow loads of 16 bytes
  int splits, rows;           // workgroups a key head's rows are dealt to, rows of one
  float* part;                // [B][H][splits][D + 2]
};
int win_step_rows(int B, int HK, int rows);
hipError_t launch_win_step(int dtype, const WinStepArgs& a, hipStream_t st);

}  // namespace kda
