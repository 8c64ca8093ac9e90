// Selective state space scan: forward, backward and single-token step.
//
// A channel's states are spread over LPC = NP / 4 neighbouring lanes, four each, and a workgroup
// holds CH = 256 / LPC channels of one group, whose B_t and C_t its lanes then share. It walks the
// tokens of one segment in chunks of 16: the chunk's inputs are loaded one chunk ahead, turned into
// dt and dt x by the lanes that loaded them, and passed through shared memory; the recurrence
// itself stays in registers. The work is bound by the vector unit, mostly by the one exponential a
// state and token needs (a quarter-rate instruction).
//
// A call with few channels and sequences is cut along the tokens too: a first pass over all
// segments but a sequence's last finds what each adds to the carried state, h_out = exp(A sum dt)
// h_in + loc, and every segment of the second pass joins those before it on entry. That runs the
// recurrence twice, so it is only done where the uncut grid leaves the chip idle (scan_seg).
#include "layer_device.h"

namespace kda {

namespace {

constexpr int TT = kScanChunk;
constexpr int NPL = kScanStates;

// The segment of a workgroup.
struct Segment {
  int n;               // sequence
  int j, count;        // place among the sequence's segments, their number
  int64_t first;       // the sequence's first segment
  int64_t t0;          // first token
  int len;             // tokens
  int64_t chunk0;      // first chunk
};

__device__ __forceinline__ Segment segment_at(const ScanArgs& a, int64_t s) {
  Segment g;
  if (a.sq.cu != nullptr) {
    g.n = find_seq(a.segoff, a.sq.n, s);
    g.first = a.segoff[g.n];
    g.count = (int)(a.segoff[g.n + 1] - g.first);
    g.chunk0 = a.choff[g.n];
  } else {
    g.count = a.sq.T > 0 ? (a.sq.T + a.seg - 1) / a.seg : 1;
    g.n = (int)(s / g.count);
    g.first = (int64_t)g.n * g.count;
    g.chunk0 = (int64_t)g.n * ((a.sq.T + TT - 1) / TT);
  }
  g.j = (int)(s - g.first);
  const int64_t begin = seq_begin(a.sq, g.n), end = seq_end(a.sq, g.n);
  g.t0 = begin + (int64_t)g.j * a.seg;
  g.len = (int)min((int64_t)a.seg, end - g.t0);
  g.chunk0 += (int64_t)g.j * (a.seg / TT);
  return g;
}

// What a workgroup's lanes are.
template <int NP>
struct Lanes {
  static constexpr int LPC = NP / NPL;   // lanes of a channel
  static constexpr int CH = 256 / LPC;   // channels of a workgroup
  static constexpr int Q = CH / 4;       // four-channel columns of a token
  static constexpr int ITEMS = (TT * Q + 255) / 256;   // four-channel pieces a thread stages
  static constexpr int BCI = (TT * NP + 255) / 256;    // elements of B (and of C) a thread stages
};

// A lane's four of a channel's N states; those behind the N-th are zero and stay zero.
template <int NP>
__device__ __forceinline__ void load_states(const float* p, int64_t row, int N, int part, bool in, float (&v)[NPL]) {
  if (N == NP) {
    const float4 r = in ? *reinterpret_cast<const float4*>(p + row * N + part * NPL) : make_float4(0.f, 0.f, 0.f, 0.f);
    v[0] = r.x;
    v[1] = r.y;
    v[2] = r.z;
    v[3] = r.w;
    return;
  }
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int n = part * NPL + i;
    v[i] = in && n < N ? p[row * N + n] : 0.f;
  }
}
template <int NP>
__device__ __forceinline__ void store_states(float* p, int64_t row, int N, int part, bool in, const float (&v)[NPL]) {
  if (!in) return;
  if (N == NP) {
    *reinterpret_cast<float4*>(p + row * N + part * NPL) = make_float4(v[0], v[1], v[2], v[3]);
    return;
  }
#pragma unroll
  for (int i = 0; i < NPL; ++i)
    if (part * NPL + i < N) p[row * N + part * NPL + i] = v[i];
}

// Forward. OUT: y, saved and final states; otherwise only what the segment adds to the state.
template <class T, int NP, bool OUT>
__global__ __launch_bounds__(256) void sscan_fwd_kernel(ScanArgs a, int tiles) {
  typedef Lanes<NP> L;
  __shared__ float2 sX[TT][L::CH];          // dt, dt x
  __shared__ float sB[TT][NP], sC[OUT ? TT : 1][NP];
  __shared__ float sY[OUT ? TT : 1][L::CH];
  const int per = a.D / a.G;                // channels of a group
  const int bx = blockIdx.x % (a.G * tiles), grp = bx / tiles;
  const int c0 = (bx % tiles) * L::CH;      // first channel, within the group
  const Segment sg = segment_at(a, blockIdx.x / (a.G * tiles));
  if (!OUT && sg.j == sg.count - 1) return;
  const int tid = threadIdx.x, part = tid % L::LPC, chl = tid / L::LPC;
  const bool in = c0 + chl < per;
  const int64_t d = (int64_t)grp * per + c0 + chl;
  const bool vec = a.vec != 0;

  float A2[NPL], h[NPL];  // exp(dt A) = 2^(dt A log2 e): the factor is folded into A once
  load_states<NP>(a.A, d, a.N, part, in, A2);
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    A2[i] *= kLog2e;
    h[i] = 0.f;
  }
  if (OUT) {
    if (a.h0 != nullptr) load_states<NP>(a.h0, (int64_t)sg.n * a.D + d, a.N, part, in, h);
    if (in)
      for (int64_t s = sg.first; s < sg.first + sg.j; ++s) {
        const float sum = a.seg_dt[s * a.D + d];
        const float4 loc = *reinterpret_cast<const float4*>(a.seg_state + (s * a.D + d) * NP + part * NPL);
        const float add[NPL] = {loc.x, loc.y, loc.z, loc.w};
#pragma unroll
        for (int i = 0; i < NPL; ++i) h[i] = fmaf(exp2_hw(sum * A2[i]), h[i], add[i]);
      }
  }
  float total = 0.f;  // sum of dt

  // staged pieces: token pt of the chunk, channels pc .. pc + 3
  float bias[L::ITEMS][4], skip[L::ITEMS][4];
  Vec<T, 4> rx[L::ITEMS], rd[L::ITEMS], rz[L::ITEMS];
  T rb[L::BCI], rc[L::BCI];
#pragma unroll
  for (int k = 0; k < L::ITEMS; ++k) {
    const int pc = c0 + (tid + k * 256) % L::Q * 4;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool ok = tid + k * 256 < TT * L::Q && pc + e < per;
      bias[k][e] = ok && a.dt_bias != nullptr ? a.dt_bias[(int64_t)grp * per + pc + e] : 0.f;
      skip[k][e] = OUT && ok && a.skip != nullptr ? a.skip[(int64_t)grp * per + pc + e] : 0.f;
    }
  }
  auto fetch = [&](int at) {  // the chunk that begins at token `at` of the segment
#pragma unroll
    for (int k = 0; k < L::ITEMS; ++k) {
      const int p = tid + k * 256, pt = at + p / L::Q, pc = c0 + p % L::Q * 4;
      const int valid = p < TT * L::Q && pt < sg.len ? per - pc : 0;
      const int64_t t = sg.t0 + pt, col = (int64_t)grp * per + pc;
      rx[k] = load_n<T, 4>(static_cast<const T*>(a.x) + t * a.x_row + col, valid, vec);
      rd[k] = load_n<T, 4>(static_cast<const T*>(a.dt) + t * a.dt_row + col, valid, vec);
      if (OUT && a.z != nullptr) rz[k] = load_n<T, 4>(static_cast<const T*>(a.z) + t * a.z_row + col, valid, vec);
    }
#pragma unroll
    for (int k = 0; k < L::BCI; ++k) {
      const int p = tid + k * 256, pt = at + p / NP, n = p % NP;
      const bool ok = p < TT * NP && pt < sg.len && n < a.N;
      const int64_t t = sg.t0 + pt;
      rb[k] = ok ? static_cast<const T*>(a.B)[t * a.b_row + (int64_t)grp * a.N + n] : (T)0.f;
      if (OUT) rc[k] = ok ? static_cast<const T*>(a.C)[t * a.c_row + (int64_t)grp * a.N + n] : (T)0.f;
    }
  };
  if (sg.len > 0) fetch(0);
  for (int at = 0; at < sg.len; at += TT) {
    Vec<T, 4> kx[L::ITEMS], kz[L::ITEMS];  // this chunk's, for its outputs
#pragma unroll
    for (int k = 0; k < L::ITEMS; ++k) {
      const int p = tid + k * 256, pt = p / L::Q;
      kx[k] = rx[k];
      kz[k] = rz[k];
      if (p < TT * L::Q) {
        // a token behind the segment's end gets dt = 0: it leaves the state as it is
        const bool live = at + pt < sg.len;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float dt = as_f(rd[k].v[e]) + bias[k][e];
          if (a.softplus) dt = softplus(dt);
          dt = live ? dt : 0.f;
          sX[pt][p % L::Q * 4 + e] = make_float2(dt, dt * as_f(rx[k].v[e]));
        }
      }
    }
#pragma unroll
    for (int k = 0; k < L::BCI; ++k) {
      const int p = tid + k * 256;
      if (p < TT * NP) {
        sB[p / NP][p % NP] = as_f(rb[k]);
        if (OUT) sC[p / NP][p % NP] = as_f(rc[k]);
      }
    }
    __syncthreads();
    if (at + TT < sg.len) fetch(at + TT);
    if (OUT && a.states != nullptr) store_states<NP>(a.states, (sg.chunk0 + at / TT) * a.D + d, a.N, part, in, h);
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const float2 v = sX[t][chl];
      const float4 b4 = *reinterpret_cast<const float4*>(&sB[t][part * NPL]);
      const float bb[NPL] = {b4.x, b4.y, b4.z, b4.w};
      float y = 0.f;
      if (!OUT) total += v.x;
#pragma unroll
      for (int i = 0; i < NPL; ++i) h[i] = fmaf(exp2_hw(v.x * A2[i]), h[i], v.y * bb[i]);
      if (OUT) {
        const float4 c4 = *reinterpret_cast<const float4*>(&sC[t][part * NPL]);
        const float cc[NPL] = {c4.x, c4.y, c4.z, c4.w};
#pragma unroll
        for (int i = 0; i < NPL; ++i) y = fmaf(cc[i], h[i], y);
        y = group_sum<L::LPC>(y);
        if (part == 0) sY[t][chl] = y;
      }
    }
    __syncthreads();
    if (OUT) {
#pragma unroll
      for (int k = 0; k < L::ITEMS; ++k) {
        const int p = tid + k * 256, pt = p / L::Q, pc = p % L::Q * 4;
        if (p < TT * L::Q && at + pt < sg.len) {
          float out[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            out[e] = fmaf(skip[k][e], as_f(kx[k].v[e]), sY[pt][pc + e]);
            if (a.z != nullptr) {
              const float z = as_f(kz[k].v[e]);
              out[e] *= z * sigmoid(z);
            }
          }
          store_n<T, 4>(static_cast<T*>(a.y) + (sg.t0 + at + pt) * a.D + (int64_t)grp * per + c0 + pc, out, per - c0 - pc, vec);
        }
      }
    }
  }
  if (OUT) {
    if (a.final_state != nullptr && sg.j == sg.count - 1)
      store_states<NP>(a.final_state, (int64_t)sg.n * a.D + d, a.N, part, in, h);
  } else if (in) {
    const int64_t s = sg.first + sg.j;
    if (part == 0) a.seg_dt[s * a.D + d] = total;
    *reinterpret_cast<float4*>(a.seg_state + (s * a.D + d) * NP + part * NPL) = make_float4(h[0], h[1], h[2], h[3]);
  }
}

// What a segment adds to the gradient of the state that enters it, for all segments but a
// sequence's first: q = a_t r_t with r_t = C_t dy'_t + q_{t+1}, walked in reverse from q = 0, and the
// sum of dt.
template <class T, int NP>
__global__ __launch_bounds__(256) void sscan_bwd_local_kernel(ScanArgs a, int tiles) {
  typedef Lanes<NP> L;
  __shared__ float2 sX[TT][L::CH];          // dt, dy'
  __shared__ float sC[TT][NP];
  const int per = a.D / a.G;
  const int bx = blockIdx.x % (a.G * tiles), grp = bx / tiles;
  const int c0 = (bx % tiles) * L::CH;
  const Segment sg = segment_at(a, blockIdx.x / (a.G * tiles));
  if (sg.j == 0) return;
  const int tid = threadIdx.x, part = tid % L::LPC, chl = tid / L::LPC;
  const bool in = c0 + chl < per;
  const int64_t d = (int64_t)grp * per + c0 + chl;
  const bool vec = a.vec != 0;
  float A2[NPL], q[NPL];
  load_states<NP>(a.A, d, a.N, part, in, A2);
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    A2[i] *= kLog2e;
    q[i] = 0.f;
  }
  float total = 0.f;
  float bias[L::ITEMS][4];
  Vec<T, 4> rd[L::ITEMS], rz[L::ITEMS], ry[L::ITEMS];
  T rc[L::BCI];
#pragma unroll
  for (int k = 0; k < L::ITEMS; ++k) {
    const int pc = c0 + (tid + k * 256) % L::Q * 4;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool ok = tid + k * 256 < TT * L::Q && pc + e < per;
      bias[k][e] = ok && a.dt_bias != nullptr ? a.dt_bias[(int64_t)grp * per + pc + e] : 0.f;
    }
  }
  auto fetch = [&](int at) {
#pragma unroll
    for (int k = 0; k < L::ITEMS; ++k) {
      const int p = tid + k * 256, pt = at + p / L::Q, pc = c0 + p % L::Q * 4;
      const int valid = p < TT * L::Q && pt < sg.len ? per - pc : 0;
      const int64_t t = sg.t0 + pt, col = (int64_t)grp * per + pc;
      rd[k] = load_n<T, 4>(static_cast<const T*>(a.dt) + t * a.dt_row + col, valid, vec);
      ry[k] = load_n<T, 4>(static_cast<const T*>(a.dy) + t * a.D + col, valid, vec);
      if (a.z != nullptr) rz[k] = load_n<T, 4>(static_cast<const T*>(a.z) + t * a.z_row + col, valid, vec);
    }
#pragma unroll
    for (int k = 0; k < L::BCI; ++k) {
      const int p = tid + k * 256, pt = at + p / NP, n = p % NP;
      const bool ok = p < TT * NP && pt < sg.len && n < a.N;
      rc[k] = ok ? static_cast<const T*>(a.C)[(sg.t0 + pt) * a.c_row + (int64_t)grp * a.N + n] : (T)0.f;
    }
  };
  const int last = (sg.len - 1) / TT * TT;
  if (sg.len > 0) fetch(last);
  for (int at = last; at >= 0 && sg.len > 0; at -= TT) {
#pragma unroll
    for (int k = 0; k < L::ITEMS; ++k) {
      const int p = tid + k * 256, pt = p / L::Q;
      if (p < TT * L::Q) {
        const bool live = at + pt < sg.len;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float dt = as_f(rd[k].v[e]) + bias[k][e];
          if (a.softplus) dt = softplus(dt);
          float g = as_f(ry[k].v[e]);
          if (a.z != nullptr) {
            const float z = as_f(rz[k].v[e]);
            g *= z * sigmoid(z);
          }
          sX[pt][p % L::Q * 4 + e] = make_float2(live ? dt : 0.f, live ? g : 0.f);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < L::BCI; ++k) {
      const int p = tid + k * 256;
      if (p < TT * NP) sC[p / NP][p % NP] = as_f(rc[k]);
    }
    __syncthreads();
    if (at > 0) fetch(at - TT);
#pragma unroll
    for (int t = TT - 1; t >= 0; --t) {
      const float2 v = sX[t][chl];
      const float4 c4 = *reinterpret_cast<const float4*>(&sC[t][part * NPL]);
      const float cc[NPL] = {c4.x, c4.y, c4.z, c4.w};
      total += v.x;
#pragma unroll
      for (int i = 0; i < NPL; ++i) q[i] = exp2_hw(v.x * A2[i]) * fmaf(cc[i], v.y, q[i]);
    }
    __syncthreads();
  }
  if (in) {
    const int64_t s = sg.first + sg.j;
    if (part == 0) a.seg_dt[s * a.D + d] = total;
    *reinterpret_cast<float4*>(a.seg_state + (s * a.D + d) * NP + part * NPL) = make_float4(q[0], q[1], q[2], q[3]);
  }
}

// Pairs of values whose lanes differ in bit D: a lane keeps the first value's sum over the pair of
// lanes where its bit is clear, the second's where it is set.
template <int D>
__device__ __forceinline__ float merge(float x, float y, int lane) {
  if constexpr (D == 32) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(y), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  if constexpr (D == 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(y), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  if constexpr (D < 16) {
    const bool up = lane & D;
    const float keep = up ? y : x, give = up ? x : y;
    return keep + xor_lane<D>(give);
  }
}

// Backward of a segment, chunk by chunk from its end. From the saved state that enters a chunk the
// 16 states and decays are formed again into registers; then, in reverse, with dy' = dy silu(z),
//   r = C dy' + q,   q <- a r,   p = q h_{t-1},
//   dC += dy' h (summed over the group's channels),  dB += r dt x,  dA += dt p,
//   dx = dt sum_n r B + skip dy',   ddt = x sum_n r B + sum_n A p,   dz = dy y' silu'(z).
// The sums over channels are joined over the wave's lanes by merges (half the values move at each
// step), over the four waves in shared memory, and over channel tiles by a second kernel.
template <class T, int NP>
__global__ __launch_bounds__(256) void sscan_bwd_kernel(ScanArgs a, int tiles) {
  typedef Lanes<NP> L;
  constexpr int LEFT = L::LPC >= 16 ? 2 : 1;  // of 8 values, what a lane ends with: the wave has 64 / LPC channels
  __shared__ float2 sX[TT][L::CH];          // dt, dt x
  __shared__ float sG[TT][L::CH];           // dy'; then sum_n r B
  __shared__ float sP[TT][L::CH];           // y without the gate; then sum_n A p
  __shared__ float sB[TT][NP], sC[TT][NP];
  __shared__ float sS[4][TT][2 * NP];       // a wave's dC (first NP), dB
  const int per = a.D / a.G;
  const int bx = blockIdx.x % (a.G * tiles), grp = bx / tiles, tile = bx % tiles;
  const int c0 = tile * L::CH;
  const Segment sg = segment_at(a, blockIdx.x / (a.G * tiles));
  const int tid = threadIdx.x, part = tid % L::LPC, chl = tid / L::LPC, lane = tid % 64, wave = tid / 64;
  const bool in = c0 + chl < per;
  const int64_t d = (int64_t)grp * per + c0 + chl;
  const bool vec = a.vec != 0;
  float A[NPL], q[NPL], dA[NPL];
  load_states<NP>(a.A, d, a.N, part, in, A);
#pragma unroll
  for (int i = 0; i < NPL; ++i) q[i] = dA[i] = 0.f;
  if (a.dfinal != nullptr) load_states<NP>(a.dfinal, (int64_t)sg.n * a.D + d, a.N, part, in, q);
  if (in)
    for (int64_t s = sg.first + sg.count - 1; s > sg.first + sg.j; --s) {
      const float sum = a.seg_dt[s * a.D + d];
      const float4 loc = *reinterpret_cast<const float4*>(a.seg_state + (s * a.D + d) * NP + part * NPL);
      const float add[NPL] = {loc.x, loc.y, loc.z, loc.w};
#pragma unroll
      for (int i = 0; i < NPL; ++i) q[i] = fmaf(exp2_hw(sum * (A[i] * kLog2e)), q[i], add[i]);
    }
  float bias[L::ITEMS][4], skip[L::ITEMS][4], dskip[L::ITEMS][4], dbias[L::ITEMS][4];
  Vec<T, 4> rx[L::ITEMS], rd[L::ITEMS], rz[L::ITEMS], ry[L::ITEMS];
  T rb[L::BCI], rc[L::BCI];
  float nh[NPL];
#pragma unroll
  for (int k = 0; k < L::ITEMS; ++k) {
    const int pc = c0 + (tid + k * 256) % L::Q * 4;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool ok = tid + k * 256 < TT * L::Q && pc + e < per;
      bias[k][e] = ok && a.dt_bias != nullptr ? a.dt_bias[(int64_t)grp * per + pc + e] : 0.f;
      skip[k][e] = ok && a.skip != nullptr ? a.skip[(int64_t)grp * per + pc + e] : 0.f;
      dskip[k][e] = dbias[k][e] = 0.f;
    }
  }
  auto fetch = [&](int at) {
#pragma unroll
    for (int k = 0; k < L::ITEMS; ++k) {
      const int p = tid + k * 256, pt = at + p / L::Q, pc = c0 + p % L::Q * 4;
      const int valid = p < TT * L::Q && pt < sg.len ? per - pc : 0;
      const int64_t t = sg.t0 + pt, col = (int64_t)grp * per + pc;
      rx[k] = load_n<T, 4>(static_cast<const T*>(a.x) + t * a.x_row + col, valid, vec);
      rd[k] = load_n<T, 4>(static_cast<const T*>(a.dt) + t * a.dt_row + col, valid, vec);
      ry[k] = load_n<T, 4>(static_cast<const T*>(a.dy) + t * a.D + col, valid, vec);
      if (a.z != nullptr) rz[k] = load_n<T, 4>(static_cast<const T*>(a.z) + t * a.z_row + col, valid, vec);
    }
#pragma unroll
    for (int k = 0; k < L::BCI; ++k) {
      const int p = tid + k * 256, pt = at + p / NP, n = p % NP;
      const bool ok = p < TT * NP && pt < sg.len && n < a.N;
      const int64_t t = sg.t0 + pt;
      rb[k] = ok ? static_cast<const T*>(a.B)[t * a.b_row + (int64_t)grp * a.N + n] : (T)0.f;
      rc[k] = ok ? static_cast<const T*>(a.C)[t * a.c_row + (int64_t)grp * a.N + n] : (T)0.f;
    }
    load_states<NP>(a.states, (sg.chunk0 + at / TT) * a.D + d, a.N, part, in, nh);
  };
  const int last = (sg.len - 1) / TT * TT;
  if (sg.len > 0) fetch(last);
  for (int at = last; at >= 0 && sg.len > 0; at -= TT) {
    Vec<T, 4> kx[L::ITEMS], kd[L::ITEMS], kz[L::ITEMS], ky[L::ITEMS];
    float hs[TT + 1][NPL], as[TT][NPL];
#pragma unroll
    for (int k = 0; k < L::ITEMS; ++k) {
      const int p = tid + k * 256, pt = p / L::Q;
      kx[k] = rx[k];
      kd[k] = rd[k];
      kz[k] = rz[k];
      ky[k] = ry[k];
      if (p < TT * L::Q) {
        const bool live = at + pt < sg.len;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float dt = as_f(rd[k].v[e]) + bias[k][e];
          if (a.softplus) dt = softplus(dt);
          dt = live ? dt : 0.f;
          float g = as_f(ry[k].v[e]);
          if (a.z != nullptr) {
            const float z = as_f(rz[k].v[e]);
            g *= z * sigmoid(z);
          }
          sX[pt][p % L::Q * 4 + e] = make_float2(dt, dt * as_f(rx[k].v[e]));
          sG[pt][p % L::Q * 4 + e] = g;
        }
      }
    }
#pragma unroll
    for (int k = 0; k < L::BCI; ++k) {
      const int p = tid + k * 256;
      if (p < TT * NP) {
        sB[p / NP][p % NP] = as_f(rb[k]);
        sC[p / NP][p % NP] = as_f(rc[k]);
      }
    }
#pragma unroll
    for (int i = 0; i < NPL; ++i) hs[0][i] = nh[i];
    __syncthreads();
    if (at > 0) fetch(at - TT);
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const float2 v = sX[t][chl];
      const float4 b4 = *reinterpret_cast<const float4*>(&sB[t][part * NPL]);
      const float bb[NPL] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        as[t][i] = exp2_hw(v.x * (A[i] * kLog2e));
        hs[t + 1][i] = fmaf(as[t][i], hs[t][i], v.y * bb[i]);
      }
      if (a.z != nullptr) {
        const float4 c4 = *reinterpret_cast<const float4*>(&sC[t][part * NPL]);
        float y = fmaf(c4.x, hs[t + 1][0], fmaf(c4.y, hs[t + 1][1], fmaf(c4.z, hs[t + 1][2], c4.w * hs[t + 1][3])));
        y = group_sum<L::LPC>(y);
        if (part == 0) sP[t][chl] = y;
      }
    }
    if (a.z != nullptr) {
      // dz needs y before sP is used again
      __syncthreads();
#pragma unroll
      for (int k = 0; k < L::ITEMS; ++k) {
        const int p = tid + k * 256, pt = p / L::Q, pc = p % L::Q * 4;
        if (p < TT * L::Q && at + pt < sg.len) {
          float out[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float z = as_f(kz[k].v[e]), s = sigmoid(z);
            out[e] = as_f(ky[k].v[e]) * fmaf(skip[k][e], as_f(kx[k].v[e]), sP[pt][pc + e]) * (s * (1.f + z * (1.f - s)));
          }
          if (a.dz != nullptr)
            store_n<T, 4>(static_cast<T*>(a.dz) + (sg.t0 + at + pt) * a.D + (int64_t)grp * per + c0 + pc, out, per - c0 - pc, vec);
        }
      }
      __syncthreads();
    }
    float dAc[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i) dAc[i] = 0.f;
#pragma unroll
    for (int t = TT - 1; t >= 0; --t) {
      const float2 v = sX[t][chl];
      const float g = sG[t][chl];
      const float4 b4 = *reinterpret_cast<const float4*>(&sB[t][part * NPL]);
      const float4 c4 = *reinterpret_cast<const float4*>(&sC[t][part * NPL]);
      const float bb[NPL] = {b4.x, b4.y, b4.z, b4.w}, cc[NPL] = {c4.x, c4.y, c4.z, c4.w};
      float s1 = 0.f, s2 = 0.f, val[8];
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        const float r = fmaf(cc[i], g, q[i]);
        val[i] = g * hs[t + 1][i];
        val[4 + i] = r * v.y;
        s1 = fmaf(r, bb[i], s1);
        q[i] = as[t][i] * r;
        const float p = q[i] * hs[t][i];
        s2 = fmaf(p, A[i], s2);
        dAc[i] = fmaf(p, v.x, dAc[i]);
      }
      s1 = group_sum<L::LPC>(s1);
      s2 = group_sum<L::LPC>(s2);
      if (part == 0) {
        sG[t][chl] = s1;  // this lane group alone reads and writes its channel's place
        sP[t][chl] = s2;
      }
      // val[0..3]: dC, val[4..7]: dB of this lane's four states; lanes of the wave with the same part
      // hold the other channels
      float m4[4], m2[2];
#pragma unroll
      for (int i = 0; i < 4; ++i) m4[i] = merge<32>(val[i], val[4 + i], lane);   // bit 5: dC or dB
#pragma unroll
      for (int i = 0; i < 2; ++i) m2[i] = merge<16>(m4[i], m4[2 + i], lane);     // bit 4: states 0, 1 or 2, 3
      const int kind = lane >> 5, pair = (lane >> 4) & 1;
      float* to = &sS[wave][t][kind * NP + part * NPL + pair * 2];
      if constexpr (LEFT == 2) {
        // LPC = 16: two values left, every lane's own
        to[0] = m2[0];
        to[1] = m2[1];
      } else {
        float m = merge<8>(m2[0], m2[1], lane);                                  // bit 3: the one or the other
        if constexpr (L::LPC <= 4) m += xor_lane<4>(m);
        if constexpr (L::LPC <= 2) m += xor_lane<2>(m);
        if constexpr (L::LPC <= 1) m += xor_lane<1>(m);
        if ((lane & 7) < L::LPC) to[(lane >> 3) & 1] = m;
      }
    }
#pragma unroll
    for (int i = 0; i < NPL; ++i) dA[i] += dAc[i];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < L::ITEMS; ++k) {
      const int p = tid + k * 256, pt = p / L::Q, pc = p % L::Q * 4;
      if (p < TT * L::Q && at + pt < sg.len) {
        float ox[4], od[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float raw = as_f(kd[k].v[e]) + bias[k][e], x = as_f(kx[k].v[e]);
          float g = as_f(ky[k].v[e]);
          if (a.z != nullptr) {
            const float z = as_f(kz[k].v[e]);
            g *= z * sigmoid(z);
          }
          const float s1 = sG[pt][pc + e];
          ox[e] = fmaf(sX[pt][pc + e].x, s1, skip[k][e] * g);
          od[e] = fmaf(x, s1, sP[pt][pc + e]);
          if (a.softplus) od[e] *= sigmoid(raw);
          dskip[k][e] = fmaf(g, x, dskip[k][e]);
          dbias[k][e] += od[e];
        }
        const int64_t o = (sg.t0 + at + pt) * a.D + (int64_t)grp * per + c0 + pc;
        store_n<T, 4>(static_cast<T*>(a.dx) + o, ox, per - c0 - pc, vec);
        store_n<T, 4>(static_cast<T*>(a.ddt) + o, od, per - c0 - pc, vec);
      }
    }
    for (int p = tid; p < TT * 2 * NP; p += 256) {
      const int pt = p / (2 * NP), v = p % (2 * NP);
      if (at + pt < sg.len)
        a.part_bc[(((int64_t)tile * a.sq.total + sg.t0 + at + pt) * a.G + grp) * 2 * NP + v] =
            (sS[0][pt][v] + sS[1][pt][v]) + (sS[2][pt][v] + sS[3][pt][v]);
    }
    __syncthreads();
  }
  const int64_t s = sg.first + sg.j;
  if (a.dh0 != nullptr && sg.j == 0) store_states<NP>(a.dh0, (int64_t)sg.n * a.D + d, a.N, part, in, q);
  if (in) *reinterpret_cast<float4*>(a.part_a + (s * a.D + d) * NP + part * NPL) = make_float4(dA[0], dA[1], dA[2], dA[3]);
  // dskip and ddt_bias: the 16 (or fewer) threads that staged a channel join in shared memory
  for (int which = 0; which < 2; ++which) {
    __syncthreads();
#pragma unroll
    for (int k = 0; k < L::ITEMS; ++k) {
      const int p = tid + k * 256;
      if (p < TT * L::Q)
#pragma unroll
        for (int e = 0; e < 4; ++e) sG[p / L::Q][p % L::Q * 4 + e] = which == 0 ? dskip[k][e] : dbias[k][e];
    }
    __syncthreads();
    if (tid < L::CH && c0 + tid < per) {
      float sum = 0.f;
#pragma unroll
      for (int t = 0; t < TT; ++t) sum += sG[t][tid];
      a.part_d[(s * 2 + which) * a.D + (int64_t)grp * per + c0 + tid] = sum;
    }
  }
}

// dB and dC from the channel tiles' sums.
template <class T, int NP>
__global__ __launch_bounds__(256) void sscan_bc_kernel(ScanArgs a, int tiles) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;  // (token, group, state)
  const int64_t rows = a.sq.total * a.G;
  if (i >= rows * a.N) return;
  const int64_t row = i / a.N;
  const int n = (int)(i % a.N);
  float c = 0.f, b = 0.f;
  for (int t = 0; t < tiles; ++t) {
    const float* p = a.part_bc + ((int64_t)t * rows + row) * 2 * NP;
    c += p[n];
    b += p[NP + n];
  }
  static_cast<T*>(a.dC)[i] = (T)c;
  static_cast<T*>(a.dB)[i] = (T)b;
}

// dA [D][N], dskip [D], ddt_bias [D] from the segments' sums: 64 columns a workgroup, the segments
// dealt to 4 lanes a column.
__global__ __launch_bounds__(256) void sscan_param_kernel(ScanArgs a, int NP) {
  __shared__ float sh[4][64];
  const int tx = threadIdx.x % 64, ty = threadIdx.x / 64;
  const int64_t col = (int64_t)blockIdx.x * 64 + tx, na = (int64_t)a.D * NP, cols = na + 2 * (int64_t)a.D;
  const float* p = col < na ? a.part_a + col : a.part_d + (col - na);
  const int64_t stride = col < na ? na : 2 * (int64_t)a.D;
  float s = 0.f;
  if (col < cols)
    for (int64_t r = ty; r < a.nseg; r += 4) s += p[r * stride];
  sh[ty][tx] = s;
  __syncthreads();
  if (ty != 0 || col >= cols) return;
  s = (sh[0][tx] + sh[1][tx]) + (sh[2][tx] + sh[3][tx]);
  if (col < na) {
    if (col % NP < a.N) a.dA[col / NP * a.N + col % NP] = s;
  } else if (col < na + a.D) {
    if (a.dskip != nullptr) a.dskip[col - na] = s;
  } else if (a.ddt_bias != nullptr) {
    a.ddt_bias[col - na - a.D] = s;
  }
}

// First segment and first chunk of each packed sequence.
__global__ __launch_bounds__(1024) void sscan_tables_kernel(const int32_t* cu, int n, int seg, int32_t* segoff,
                                                            int32_t* choff) {
  __shared__ int sh[2][1024];
  int base[2] = {0, 0};
  for (int i0 = 0; i0 < n; i0 += 1024) {
    const int i = i0 + threadIdx.x;
    const int len = i < n ? cu[i + 1] - cu[i] : 0;
    const int mine[2] = {i < n ? max(1, (len + seg - 1) / seg) : 0, i < n ? (len + TT - 1) / TT : 0};
    sh[0][threadIdx.x] = mine[0];
    sh[1][threadIdx.x] = mine[1];
    __syncthreads();
    for (int step = 1; step < 1024; step *= 2) {
      int add[2] = {0, 0};
      if ((int)threadIdx.x >= step) {
        add[0] = sh[0][threadIdx.x - step];
        add[1] = sh[1][threadIdx.x - step];
      }
      __syncthreads();
      sh[0][threadIdx.x] += add[0];
      sh[1][threadIdx.x] += add[1];
      __syncthreads();
    }
    if (i < n) {
      segoff[i] = base[0] + sh[0][threadIdx.x] - mine[0];
      choff[i] = base[1] + sh[1][threadIdx.x] - mine[1];
    }
    base[0] += sh[0][1023];
    base[1] += sh[1][1023];
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    segoff[n] = base[0];
    choff[n] = base[1];
  }
}

// One token: lanes as in the scan, the state read and written in place.
template <class T, int NP>
__global__ __launch_bounds__(256) void sscan_step_kernel(ScanStepArgs a, int tiles) {
  typedef Lanes<NP> L;
  const int per = a.D / a.G;
  const int grp = blockIdx.x / tiles, c0 = blockIdx.x % tiles * L::CH, b = blockIdx.y;
  const int part = threadIdx.x % L::LPC, chl = threadIdx.x / L::LPC;
  const int slot = step_slot(a.slots, b, a.slots_n);
  const bool in = c0 + chl < per;
  const int64_t d = (int64_t)grp * per + c0 + chl;
  if (!in) return;
  T* y = static_cast<T*>(a.y) + (int64_t)b * a.D + d;
  if (slot < 0) {
    if (part == 0) *y = (T)(slot == -1 ? 0.f : __builtin_nanf(""));
    return;
  }
  float h[NPL], A[NPL];
  const int64_t row = (int64_t)slot * a.D + d;
  load_states<NP>(a.state, row, a.N, part, true, h);
  load_states<NP>(a.A, d, a.N, part, true, A);
  const float x = as_f(static_cast<const T*>(a.x)[b * a.x_row + d]);
  float dt = as_f(static_cast<const T*>(a.dt)[b * a.dt_row + d]) + (a.dt_bias != nullptr ? a.dt_bias[d] : 0.f);
  if (a.softplus) dt = softplus(dt);
  const T* Bm = static_cast<const T*>(a.Bm) + b * a.b_row + (int64_t)grp * a.N;
  const T* Cm = static_cast<const T*>(a.Cm) + b * a.c_row + (int64_t)grp * a.N;
  float out = 0.f;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int n = part * NPL + i;
    const bool ok = n < a.N;
    h[i] = fmaf(exp2_hw(dt * (A[i] * kLog2e)), h[i], dt * x * (ok ? as_f(Bm[n]) : 0.f));
    out = fmaf(ok ? as_f(Cm[n]) : 0.f, h[i], out);
  }
  store_states<NP>(a.state, row, a.N, part, true, h);
  out = group_sum<L::LPC>(out);
  if (part == 0) {
    if (a.skip != nullptr) out = fmaf(a.skip[d], x, out);
    if (a.z != nullptr) {
      const float z = as_f(static_cast<const T*>(a.z)[b * a.z_row + d]);
      out *= z * sigmoid(z);
    }
    *y = (T)out;
  }
}

template <class T, int NP>
hipError_t fwd_np(const ScanArgs& a, hipStream_t st) {
  const int tiles = scan_tiles(a.D, a.N, a.G);
  const dim3 grid((unsigned)(a.nseg * a.G * tiles));
  if (a.split) {
    hipLaunchKernelGGL((sscan_fwd_kernel<T, NP, false>), grid, dim3(256), 0, st, a, tiles);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((sscan_fwd_kernel<T, NP, true>), grid, dim3(256), 0, st, a, tiles);
  return hipGetLastError();
}

template <class T, int NP>
hipError_t bwd_np(const ScanArgs& a, hipStream_t st) {
  const int tiles = scan_tiles(a.D, a.N, a.G);
  const dim3 grid((unsigned)(a.nseg * a.G * tiles));
  hipError_t e;
  if (a.split) {
    hipLaunchKernelGGL((sscan_bwd_local_kernel<T, NP>), grid, dim3(256), 0, st, a, tiles);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  hipLaunchKernelGGL((sscan_bwd_kernel<T, NP>), grid, dim3(256), 0, st, a, tiles);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  const int64_t bc = a.sq.total * a.G * a.N;
  if (bc > 0) {
    hipLaunchKernelGGL((sscan_bc_kernel<T, NP>), dim3((unsigned)((bc + 255) / 256)), dim3(256), 0, st, a, tiles);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  hipLaunchKernelGGL(sscan_param_kernel, dim3((unsigned)(((int64_t)a.D * (NP + 2) + 63) / 64)), dim3(256), 0, st, a, NP);
  return hipGetLastError();
}

template <class T, int NP>
hipError_t step_np(const ScanStepArgs& a, hipStream_t st) {
  const int tiles = scan_tiles(a.D, a.N, a.G);
  hipLaunchKernelGGL((sscan_step_kernel<T, NP>), dim3(tiles * a.G, a.B), dim3(256), 0, st, a, tiles);
  return hipGetLastError();
}

#define SSCAN_DISPATCH(FN)                                                       \
  do {                                                                           \
    const int np = scan_np(a.N);                                                 \
    if (dtype == KDA_F32) {                                                      \
      if (np == 8) return FN<float, 8>(a, st);                                   \
      if (np == 16) return FN<float, 16>(a, st);                                 \
      if (np == 32) return FN<float, 32>(a, st);                                 \
      return FN<float, 64>(a, st);                                               \
    }                                                                            \
    if (np == 8) return FN<bf16, 8>(a, st);                                      \
    if (np == 16) return FN<bf16, 16>(a, st);                                    \
    if (np == 32) return FN<bf16, 32>(a, st);                                    \
    return FN<bf16, 64>(a, st);                                                  \
  } while (0)

}  // namespace

int scan_np(int N) { return N <= 8 ? 8 : N <= 16 ? 16 : N <= 32 ? 32 : 64; }

int scan_tiles(int D, int N, int G) {
  const int ch = 256 / (scan_np(N) / kScanStates);
  return (D / G + ch - 1) / ch;
}

// Tokens of a segment: a cut into about four workgroups a CU (forward) or two (backward, whose
// registers allow no more), none shorter than 64 tokens. Where the longest sequence is at most two
// such segments nothing is cut: the pass that a cut needs costs more than the fuller grid gives.
int scan_seg(const Seqs& s, int64_t longest, int D, int N, int G, bool bwd) {
  const int64_t cols = (int64_t)G * scan_tiles(D, N, G);
  const int64_t whole = longest > 0 ? (longest + kScanChunk - 1) / kScanChunk * kScanChunk : kScanChunk;
  const int64_t want = bwd ? 512 : 1024;
  int64_t seg = (s.total * cols + want - 1) / want;
  seg = (seg + kScanChunk - 1) / kScanChunk * kScanChunk;
  if (seg < 64) seg = 64;
  return (int)(whole <= 2 * seg ? whole : seg);
}

hipError_t launch_scan_tables(const Seqs& s, int seg, int32_t* segoff, int32_t* choff, hipStream_t st) {
  hipLaunchKernelGGL(sscan_tables_kernel, dim3(1), dim3(1024), 0, st, s.cu, s.n, seg, segoff, choff);
  return hipGetLastError();
}

hipError_t launch_sscan_fwd(int dtype, const ScanArgs& a, hipStream_t st) { SSCAN_DISPATCH(fwd_np); }
hipError_t launch_sscan_bwd(int dtype, const ScanArgs& a, hipStream_t st) { SSCAN_DISPATCH(bwd_np); }
hipError_t launch_sscan_step(int dtype, const ScanStepArgs& a, hipStream_t st) { SSCAN_DISPATCH(step_np); }

}  // namespace kda
