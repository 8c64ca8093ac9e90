// Host-side launchers and argument blocks of the layer operators (internal to the library):
// short convolution, selective scan, group norm, KDA token step.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kda_layers.h"

namespace kda {

// Sequences on the token axis: n dense ones of T tokens, or packed ones cut at cu.
struct Seqs {
  const int32_t* cu;  // device [n + 1], or nullptr when dense
  int n;
  int T;              // tokens of a dense sequence
  int64_t total;      // tokens in all
};

struct ConvArgs {
  Seqs sq;
  int D, W, act;      // act: kda_act
  int64_t x_row;      // elements between two tokens of x
  const void *x, *h0, *dy, *dfinal;
  const float *w, *bias;
  void *y, *dx, *dh0, *final_state;
  float *dw, *db;
  float* part;        // bwd: [row blocks][W + 1][D] sums of a block's tokens
  int tt;             // tokens that a thread walks
  int vec;            // 4: rows are aligned for four elements a load; 1: they are not
  int wvec;           // weight is 16-byte aligned
};
int conv_vec(int dtype, int D, int64_t x_row, const void* const* ptrs, int np);
int conv_tile(int64_t total, int D, int vec);
int64_t conv_row_blocks(const ConvArgs& a);
hipError_t launch_conv_fwd(int dtype, const ConvArgs& a, hipStream_t st);
hipError_t launch_conv_bwd(int dtype, const ConvArgs& a, hipStream_t st);

struct ConvStepArgs {
  int B, D, W, act, slots_n, wvec;
  int64_t x_row;
  const void* x;
  const float *w, *bias;
  const int32_t* slots;
  void *state, *y;
};
hipError_t launch_conv_step(int dtype, const ConvStepArgs& a, hipStream_t st);

// States a lane holds; a channel's states (N, padded to NP) are spread over NP / 4 lanes.
constexpr int kScanStates = 4;
// Tokens of a chunk: the forward saves the state entering each, the backward walks them in reverse.
constexpr int kScanChunk = KDA_SCAN_CHUNK;
// Packed sequences that a wave counts by itself; more have tables in the workspace.
constexpr int kScanLanes = 64;

struct ScanArgs {
  Seqs sq;
  int D, N, G;
  int softplus;
  int64_t x_row, dt_row, z_row, b_row, c_row;
  const void *x, *dt, *z, *B, *C, *dy;
  const float *A, *skip, *dt_bias, *h0, *dfinal;
  void *y, *dx, *ddt, *dz, *dB, *dC;
  float *final_state, *states, *dh0, *dA, *dskip, *ddt_bias;
  // segments: every sequence is cut into max(1, ceil(len / seg)) runs of seg tokens
  int seg;                  // tokens of a segment (a multiple of the chunk)
  int64_t nseg;             // segments in all
  const int32_t* segoff;    // more than kScanLanes packed: [n + 1] first segment of each sequence
  const int32_t* choff;     // likewise its first chunk
  int split;                // some sequence has more than one segment
  int lseg;                 // tokens of a local segment (divides seg)
  int64_t nloc;             // local segments in all
  const int32_t* loff;      // likewise its first local segment
  float* seg_dt;            // [nloc][D] sum of dt over the local segment
  float* seg_state;         // [nloc][D][NP] what the local segment adds to the carried state
  float* part_bc;           // bwd [tiles of a group][tokens][G][2 NP]
  float* part_a;            // bwd [nseg][D][NP]
  float* part_d;            // bwd [nseg][2][D]: dskip, ddt_bias
  int vec;                  // rows allow four-element loads
  int bcvec;                // rows of dB and dC allow four-element stores
};
int scan_np(int N);                      // padded states
int scan_tiles(int D, int N, int G);     // channel tiles of one group
void scan_seg(const Seqs& s, int64_t longest, int D, int N, int G, bool bwd, int* seg, int* lseg);
hipError_t launch_scan_tables(const Seqs& s, int seg, int lseg, int32_t* segoff, int32_t* loff, int32_t* choff,
                              hipStream_t st);
hipError_t launch_sscan_fwd(int dtype, const ScanArgs& a, hipStream_t st);
hipError_t launch_sscan_bwd(int dtype, const ScanArgs& a, hipStream_t st);

struct ScanStepArgs {
  int B, D, N, G, softplus, slots_n;
  int64_t x_row, dt_row, z_row, b_row, c_row;
  const void *x, *dt, *z, *Bm, *Cm;
  const float *A, *skip, *dt_bias;
  const int32_t* slots;
  float* state;
  void* y;
};
hipError_t launch_sscan_step(int dtype, const ScanStepArgs& a, hipStream_t st);

struct NormArgs {
  int64_t R;
  int G, C;
  int center, act, shared;
  float eps;
  int64_t x_row, gate_row;
  const void *x, *gate, *dy;
  const float *w, *bias;
  void *y, *dx, *dgate;
  float *dw, *db;
  float* part;     // bwd [rows of sums][2][columns]
  int vec;         // rows allow vector loads
  int wvec;        // weight and bias too
};
struct NormPlan {
  int tpi, nch, vec;       // lanes of a group, chunks a lane holds, elements of a chunk
  int64_t blocks;          // workgroups
  int64_t stride;          // groups of lanes that take items: a multiple of G
  int64_t part_rows;       // rows of partial sums
  int part_cols;           // columns of one of the two sums
};
bool norm_plan(int dtype, int64_t R, int G, int C, int shared, bool bwd, NormPlan* p);
hipError_t launch_norm_fwd(int dtype, const NormArgs& a, hipStream_t st);
hipError_t launch_norm_bwd(int dtype, const NormArgs& a, hipStream_t st);

struct KdaStepArgs {
  int B, H, HV, K, V, slots_n, beta_logits;
  float scale;
  const void *q, *k, *v;
  const float *g, *beta;
  const int32_t* slots;
  float* state;
  void* o;
};
hipError_t launch_kda_step(int dtype, const KdaStepArgs& a, hipStream_t st);

}  // namespace kda
