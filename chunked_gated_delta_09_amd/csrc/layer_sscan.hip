// Selective state space scan: forward, backward and single-token step.
//
// A channel's states are spread over LPC = NP / 4 neighbouring lanes, four each, and a workgroup
// holds CH = 256 / LPC channels of one group, whose B_t and C_t its lanes then share. It walks the
// tokens of one segment in chunks of 16: the chunk's inputs are loaded one chunk ahead, turned into
// dt and dt x by the lanes that loaded them, and passed through shared memory; the recurrence
// itself stays in registers. The work is bound by the vector unit: a state and token takes five
// instructions (dt A, its exponential at half rate, dt x B, two multiply-adds), a channel and token
// about 30 more shared by its lanes. Measured, bf16, N = 16, calls back to back: B=1, T=16384, D=2048 takes 96 us
// for the first pass and 139 for the second, with the vector unit issuing 82 and 85 % of the time; B=2, T=2048,
// D=2048 takes 28 and 42 us (59 and 66 %), its backward 30 (local pass, 57 %), 131 (71 %, two waves a SIMD) and 5
// (sums). A chip that was idle has a lower clock for its first 20 ms, and the same kernels take 10 to 20 % longer
// (112, 162; 31, 46, 33, 146 us); the variants named here and below were compared there.
// Staging through two buffers with one barrier a chunk took 175 us for the 165 of that time's second
// pass. All states of a channel in one lane would save the joins over lanes, and leave a quarter of the
// waves; sixteen lanes a channel would cost four joins a state.
//
// A call with few channels and sequences is cut along the tokens too: a first pass finds what each
// local segment adds to the carried state, h_out = exp(A sum dt) h_in + loc, and every segment of the
// second pass joins those before it on entry. That runs the recurrence twice, so it is only done
// where the uncut grid leaves the chip idle (scan_seg). Local segments may be shorter: the first
// pass has fewer registers, and so room for more workgroups at a time.
#include "layer_device.h"

namespace kda {

namespace {

constexpr int TT = kScanChunk;
constexpr int NPL = kScanStates;

// A run of tokens of one sequence, as a workgroup takes it.
struct Segment {
  int n;               // sequence
  int j, count;        // place among the sequence's segments of this length, their number
  int64_t first;       // the first of them
  int64_t first_local; // the sequence's first local segment (lseg tokens each)
  int64_t first_chunk; // the sequence's first chunk
  int64_t t0;          // first token
  int len;             // tokens
};

// Segments of `seg` tokens in a sequence of `len`.
__device__ __forceinline__ int segments_of(int64_t len, int seg) { return len > 0 ? (int)((len + seg - 1) / seg) : 1; }
__device__ __forceinline__ int chunks_of(int64_t len) { return (int)((len + TT - 1) / TT); }

// Segment s (LOCAL: local segment s). Of packed sequences up to 64 each wave counts their segments itself, a
// sequence a lane; more have tables from a kernel before this one (which costs a small call 4 us).
template <bool LOCAL>
__device__ __forceinline__ Segment segment_at(const ScanArgs& a, int64_t s) {
  Segment g;
  const int seg = LOCAL ? a.lseg : a.seg;
  if (a.sq.cu == nullptr) {
    g.count = segments_of(a.sq.T, seg);
    g.n = (int)(s / g.count);
    g.first = (int64_t)g.n * g.count;
    g.first_local = (int64_t)g.n * segments_of(a.sq.T, a.lseg);
    g.first_chunk = (int64_t)g.n * chunks_of(a.sq.T);
  } else if (a.sq.n > kScanLanes) {
    const int32_t* off = LOCAL ? a.loff : a.segoff;
    g.n = find_seq(off, a.sq.n, s);
    g.first = off[g.n];
    g.count = (int)(off[g.n + 1] - g.first);
    g.first_local = a.loff[g.n];
    g.first_chunk = a.choff[g.n];
  } else {
    const int lane = threadIdx.x % 64;
    const bool has = lane < a.sq.n;
    const int len = has ? a.sq.cu[lane + 1] - a.sq.cu[lane] : 0;
    const int mine[3] = {has ? segments_of(len, a.seg) : 0, has ? segments_of(len, a.lseg) : 0, has ? chunks_of(len) : 0};
    int upto[3] = {mine[0], mine[1], mine[2]};
#pragma unroll
    for (int step = 1; step < 64; step *= 2)
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        const int below = __shfl_up(upto[k], step, 64);
        if (lane >= step) upto[k] += below;
      }
    const int w = LOCAL ? 1 : 0;
    g.n = __ffsll((unsigned long long)__ballot(has && upto[w] > s)) - 1;
    const int at = __builtin_amdgcn_readfirstlane(g.n);
    g.n = at;
    g.first = __builtin_amdgcn_readlane(upto[w] - mine[w], at);
    g.count = __builtin_amdgcn_readlane(mine[w], at);
    g.first_local = __builtin_amdgcn_readlane(upto[1] - mine[1], at);
    g.first_chunk = __builtin_amdgcn_readlane(upto[2] - mine[2], at);
  }
  g.j = (int)(s - g.first);
  g.t0 = seq_begin(a.sq, g.n) + (int64_t)g.j * seg;
  g.len = (int)min((int64_t)seg, seq_end(a.sq, g.n) - g.t0);
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

__device__ __forceinline__ void unpack(const float4& v, float (&out)[4]) {
  out[0] = v.x;
  out[1] = v.y;
  out[2] = v.z;
  out[3] = v.w;
}

// h 2^e, for e of any size: over a segment 2^e alone can be past fp32 where the product is not, and is zero where h
// is. The fraction's factor is in (1/2, 1], the rest goes into the exponent; a NaN stays one.
__device__ __forceinline__ float times_exp2(float h, float e) {
  const float low = e < -1024.f ? -1024.f : e, whole = ceilf(low);
  return ldexpf(h * exp2_hw(low - whole), (int)whole);
}

// Carries h through `count` segments from `s` on (step: the one behind or before): h <- exp(A sum dt) h +
// loc. Eight segments are loaded together, since only the sums depend on each other. The factors are at most one where dt
// comes from a softplus and no A of the wave is above zero; otherwise eight with a factor that may be past fp32 are
// taken one by one, each product formed by its exponent (for all calls that took 1 % of B=1, T=16384, D=2048, N=16:
// 240 against 238 us).
template <int NP>
__device__ __forceinline__ void join_segments(const ScanArgs& a, int64_t s, int step, int64_t count, int64_t d, int part,
                                              const float (&A2)[NPL], float (&h)[NPL]) {
  bool up = a.softplus == 0;
#pragma unroll
  for (int i = 0; i < NPL; ++i) up = up || A2[i] > 0.f;
  const bool may_grow = __any(up);
  for (int64_t k = 0; k < count; k += 8) {
    float sum[8];
    float4 loc[8];
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (k + u < count) {
        const int64_t row = (s + (int64_t)step * (k + u)) * a.D + d;
        sum[u] = a.seg_dt[row];
        loc[u] = *reinterpret_cast<const float4*>(a.seg_state + row * NP + part * NPL);
      }
    if (may_grow) {
      bool past = false;
#pragma unroll
      for (int u = 0; u < 8; ++u)
#pragma unroll
        for (int i = 0; i < NPL; ++i) past = past || (k + u < count && sum[u] * A2[i] > 126.f);
      if (__any(past)) {
#pragma unroll 1
        for (int64_t v = k; v < min(k + 8, count); ++v) {
          const int64_t row = (s + (int64_t)step * v) * a.D + d;
          float add[NPL];
          unpack(*reinterpret_cast<const float4*>(a.seg_state + row * NP + part * NPL), add);
#pragma unroll
          for (int i = 0; i < NPL; ++i) h[i] = times_exp2(h[i], a.seg_dt[row] * A2[i]) + add[i];
        }
        continue;
      }
    }
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (k + u < count) {
        const float add[NPL] = {loc[u].x, loc[u].y, loc[u].z, loc[u].w};
#pragma unroll
        for (int i = 0; i < NPL; ++i) h[i] = fmaf(exp2_hw(sum[u] * A2[i]), h[i], add[i]);
      }
  }
}

// What a thread stages of a chunk: four neighbouring channels of one token (ITEMS such pieces) and
// BCI elements of B and C. Addresses are a chunk's base, the same for the workgroup, and 32-bit byte
// offsets that stay the same for all chunks.
template <class T, int NP>
struct Stage {
  typedef Lanes<NP> L;
  int tid, per, grp, c0;
  bool vec;    // four-element loads are aligned; a piece's channels then exist all or none
  bool inner;  // and all channels of the tile exist

  __device__ __forceinline__ Stage(const ScanArgs& a, int grp_, int c0_)
      : tid(threadIdx.x), per(a.D / a.G), grp(grp_), c0(c0_), vec(a.vec != 0), inner(vec && c0_ + L::CH <= a.D / a.G) {}
  // To be called once a chunk: what follows from the thread's number (places, masks, the addresses of
  // partial chunks) is formed again rather than kept in registers across the recurrence.
  __device__ __forceinline__ void renew() { asm volatile("" : "+v"(tid)); }
  __device__ __forceinline__ bool has(int k) const { return TT * L::Q >= 256 * (k + 1) || tid + k * 256 < TT * L::Q; }
  __device__ __forceinline__ int token(int k) const { return (tid + k * 256) / L::Q; }
  __device__ __forceinline__ int col(int k) const { return (tid + k * 256) % L::Q * 4; }
  __device__ __forceinline__ int bc_token(int k) const { return (tid + k * 256) / NP; }
  __device__ __forceinline__ int bc_state(int k) const { return (tid + k * 256) % NP; }
  __device__ __forceinline__ bool bc_has(int k) const { return TT * NP >= 256 * (k + 1) || tid + k * 256 < TT * NP; }
  // this thread's place from the chunk's first row on
  __device__ __forceinline__ uint32_t offset(int k, int64_t row) const {
    return (uint32_t)((token(k) * row + (int64_t)grp * per + c0 + col(k)) * (int64_t)sizeof(T));
  }
  __device__ __forceinline__ uint32_t bc_offset(int k, int64_t row, int N) const {
    return (uint32_t)((bc_token(k) * row + (int64_t)grp * N + bc_state(k)) * (int64_t)sizeof(T));
  }
  // piece k of the chunk whose first token is t and that has `live` tokens
  __device__ __forceinline__ Pack<T, 4> load(const void* p, int64_t t, int64_t row, uint32_t off, int k, int live) const {
    const T* q = reinterpret_cast<const T*>(static_cast<const char*>(p) + t * row * (int64_t)sizeof(T) + off);
    if (inner && live >= TT) {
      if (has(k)) return load_n<T, 4>(q, 4, true);
      return Pack<T, 4>{};
    }
    const int valid = has(k) && token(k) < live ? per - c0 - col(k) : 0;
    if (vec) {
      if (valid > 0) return load_n<T, 4>(q, 4, true);
      return Pack<T, 4>{};
    }
    return load_n<T, 4>(q, valid, false);
  }
  __device__ __forceinline__ T load_bc(const void* p, int64_t t, int64_t row, uint32_t off, int k, int N, int live) const {
    const T* q = reinterpret_cast<const T*>(static_cast<const char*>(p) + t * row * (int64_t)sizeof(T) + off);
    return bc_has(k) && bc_token(k) < live && bc_state(k) < N ? *q : (T)0.f;
  }
  __device__ __forceinline__ void store(void* p, int64_t t, int64_t row, uint32_t off, int k, int live,
                                        const float (&v)[4]) const {
    T* q = reinterpret_cast<T*>(static_cast<char*>(p) + t * row * (int64_t)sizeof(T) + off);
    const int valid = has(k) && token(k) < live ? per - c0 - col(k) : 0;
    if (vec) {
      if (valid > 0) store_n<T, 4>(q, v, 4, true);
    } else {
      store_n<T, 4>(q, v, valid, false);
    }
  }
  // a parameter of the tile's channels to shared memory
  __device__ __forceinline__ void params(const float* p, float* to) const {
    if (tid < L::CH) to[tid] = p != nullptr && c0 + tid < per ? p[(int64_t)grp * per + c0 + tid] : 0.f;
  }
};

// dt of four channels from the raw steps; zero for a token that is not there, which leaves states as
// they are.
template <class T>
__device__ __forceinline__ void steps_of(const Pack<T, 4>& raw, const float (&bias)[4], int soft, bool ok, float (&dt)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) dt[e] = raw.at(e) + bias[e];
  if (soft) {
#pragma unroll
    for (int e = 0; e < 4; ++e) dt[e] = softplus(dt[e]);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) dt[e] = ok ? dt[e] : 0.f;
}
// v *= silu(z)
template <class T>
__device__ __forceinline__ void gate_by(const Pack<T, 4>& gate, float (&v)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float z = gate.at(e);
    v[e] *= z * sigmoid(z);
  }
}

// The staging threads' sums of dt (16 a channel) to seg_dt of segment s; sh: [TT][CH].
template <class T, int NP>
__device__ __forceinline__ void sum_dt(const ScanArgs& a, const Stage<T, NP>& sv, const float (&total)[Lanes<NP>::ITEMS][4],
                                       float* sh, int64_t s) {
  typedef Lanes<NP> L;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < L::ITEMS; ++k)
    if (sv.has(k))
      *reinterpret_cast<float4*>(sh + sv.token(k) * L::CH + sv.col(k)) =
          make_float4(total[k][0], total[k][1], total[k][2], total[k][3]);
  __syncthreads();
  if (sv.tid < L::CH && sv.c0 + sv.tid < sv.per) {
    float sum = 0.f;
#pragma unroll
    for (int t = 0; t < TT; ++t) sum += sh[t * L::CH + sv.tid];
    a.seg_dt[s * a.D + (int64_t)sv.grp * sv.per + sv.c0 + sv.tid] = sum;
  }
}

// Forward. OUT: y, saved and final states; otherwise only what the segment adds to the state.
template <class T, int NP, bool OUT>
__global__ __launch_bounds__(256) void sscan_fwd_kernel(ScanArgs a, int tiles) {
  typedef Lanes<NP> L;
  __shared__ float2 sX[TT][L::CH];          // dt, dt x
  __shared__ float sB[TT][NP], sC[OUT ? TT : 1][NP];
  __shared__ float sY[OUT ? TT : 1][L::CH];
  __shared__ float sBias[L::CH], sSkip[L::CH];
  const int bx = blockIdx.x % (a.G * tiles), grp = bx / tiles;
  const int c0 = (bx % tiles) * L::CH;      // first channel, within the group
  const Segment sg = segment_at<!OUT>(a, blockIdx.x / (a.G * tiles));
  // the last segment of the second pass has no successor to carry its state to
  if (!OUT && sg.j >= (segments_of(seq_end(a.sq, sg.n) - seq_begin(a.sq, sg.n), a.seg) - 1) * (a.seg / a.lseg)) return;
  Stage<T, NP> sv(a, grp, c0);
  const int tid = threadIdx.x, part = tid % L::LPC, chl = tid / L::LPC;
  const bool in = c0 + chl < sv.per;
  const int64_t d = (int64_t)grp * sv.per + c0 + chl;

  float A2[NPL], h[NPL];  // exp(dt A) = 2^(dt A log2 e): the factor is folded into A once
  load_states<NP>(a.A, d, a.N, part, in, A2);
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    A2[i] *= kLog2e;
    h[i] = 0.f;
  }
  if (OUT) {
    if (a.h0 != nullptr) load_states<NP>(a.h0, (int64_t)sg.n * a.D + d, a.N, part, in, h);
    if (in && a.split)
      join_segments<NP>(a, sg.first_local, 1, (int64_t)sg.j * (a.seg / a.lseg), d, part, A2, h);
  }
  const int64_t chunk0 = sg.first_chunk + (int64_t)sg.j * (a.seg / TT);
  float total[L::ITEMS][4] = {};  // sum of dt over the tokens that this thread stages
  sv.params(a.dt_bias, sBias);
  if (OUT) sv.params(a.skip, sSkip);

  Pack<T, 4> rx[L::ITEMS], rd[L::ITEMS], rz[L::ITEMS];
  T rb[L::BCI], rc[L::BCI];
  uint32_t ox[L::ITEMS], od[L::ITEMS], oz[L::ITEMS], oy[L::ITEMS], ob[L::BCI], oc[L::BCI];
#pragma unroll
  for (int k = 0; k < L::ITEMS; ++k) {
    ox[k] = sv.offset(k, a.x_row);
    od[k] = sv.offset(k, a.dt_row);
    oz[k] = sv.offset(k, a.z_row);
    oy[k] = sv.offset(k, a.D);
  }
#pragma unroll
  for (int k = 0; k < L::BCI; ++k) {
    ob[k] = sv.bc_offset(k, a.b_row, a.N);
    oc[k] = sv.bc_offset(k, a.c_row, a.N);
  }
  auto fetch = [&](int at) {  // the chunk that begins at token `at` of the segment
    const int64_t t = sg.t0 + at;
    const int live = sg.len - at;
#pragma unroll
    for (int k = 0; k < L::ITEMS; ++k) {
      rx[k] = sv.load(a.x, t, a.x_row, ox[k], k, live);
      rd[k] = sv.load(a.dt, t, a.dt_row, od[k], k, live);
      if (OUT && a.z != nullptr) rz[k] = sv.load(a.z, t, a.z_row, oz[k], k, live);
    }
#pragma unroll
    for (int k = 0; k < L::BCI; ++k) {
      rb[k] = sv.load_bc(a.B, t, a.b_row, ob[k], k, a.N, live);
      if (OUT) rc[k] = sv.load_bc(a.C, t, a.c_row, oc[k], k, a.N, live);
    }
  };
  if (sg.len > 0) fetch(0);
  __syncthreads();
  for (int at = 0; at < sg.len; at += TT) {
    sv.renew();
    const int live = sg.len - at;
    Pack<T, 4> kx[L::ITEMS], kz[L::ITEMS];  // this chunk's, for its outputs
#pragma unroll
    for (int k = 0; k < L::ITEMS; ++k) {
      kx[k] = rx[k];
      kz[k] = rz[k];
      if (sv.has(k)) {
        const bool ok = sv.token(k) < live;
        float bias[4];
        unpack(*reinterpret_cast<const float4*>(&sBias[sv.col(k)]), bias);
        float2* to = &sX[sv.token(k)][sv.col(k)];
        steps_of(rd[k], bias, a.softplus, ok, bias);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (!OUT) total[k][e] += bias[e];
          to[e] = make_float2(bias[e], bias[e] * rx[k].at(e));
        }
      }
    }
#pragma unroll
    for (int k = 0; k < L::BCI; ++k)
      if (sv.bc_has(k)) {
        sB[sv.bc_token(k)][sv.bc_state(k)] = as_f(rb[k]);
        if (OUT) sC[sv.bc_token(k)][sv.bc_state(k)] = as_f(rc[k]);
      }
    __syncthreads();
    if (live > TT) fetch(at + TT);
    if (OUT && a.states != nullptr) store_states<NP>(a.states, (chunk0 + at / TT) * a.D + d, a.N, part, in, h);
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const float2 v = sX[t][chl];
      float bb[NPL];
      unpack(*reinterpret_cast<const float4*>(&sB[t][part * NPL]), bb);
#pragma unroll
      for (int i = 0; i < NPL; ++i) h[i] = fmaf(exp2_hw(v.x * A2[i]), h[i], v.y * bb[i]);
      if (OUT) {
        float cc[NPL];
        unpack(*reinterpret_cast<const float4*>(&sC[t][part * NPL]), cc);
        float y = cc[0] * h[0];
#pragma unroll
        for (int i = 1; i < NPL; ++i) y = fmaf(cc[i], h[i], y);
        sY[t][chl] = group_sum<L::LPC>(y);  // the same from all lanes of the channel
      }
    }
    __syncthreads();
    if (OUT) {
#pragma unroll
      for (int k = 0; k < L::ITEMS; ++k)
        if (sv.has(k)) {
          float skip[4], out[4];
          unpack(*reinterpret_cast<const float4*>(&sSkip[sv.col(k)]), skip);
          unpack(*reinterpret_cast<const float4*>(&sY[sv.token(k)][sv.col(k)]), out);
#pragma unroll
          for (int e = 0; e < 4; ++e) out[e] = fmaf(skip[e], kx[k].at(e), out[e]);
          if (a.z != nullptr) gate_by(kz[k], out);
          sv.store(a.y, sg.t0 + at, a.D, oy[k], k, live, out);
        }
    }
  }
  if (OUT) {
    if (a.final_state != nullptr && sg.j == sg.count - 1)
      store_states<NP>(a.final_state, (int64_t)sg.n * a.D + d, a.N, part, in, h);
  } else {
    const int64_t s = sg.first + sg.j;
    if (in) *reinterpret_cast<float4*>(a.seg_state + (s * a.D + d) * NP + part * NPL) = make_float4(h[0], h[1], h[2], h[3]);
    sum_dt<T, NP>(a, sv, total, reinterpret_cast<float*>(sX), s);
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
  __shared__ float sBias[L::CH];
  const int bx = blockIdx.x % (a.G * tiles), grp = bx / tiles;
  const int c0 = (bx % tiles) * L::CH;
  const Segment sg = segment_at<true>(a, blockIdx.x / (a.G * tiles));
  if (sg.j < a.seg / a.lseg) return;  // the first segment of the second pass has no predecessor
  Stage<T, NP> sv(a, grp, c0);
  const int tid = threadIdx.x, part = tid % L::LPC, chl = tid / L::LPC;
  const bool in = c0 + chl < sv.per;
  const int64_t d = (int64_t)grp * sv.per + c0 + chl;
  float A2[NPL], q[NPL];
  load_states<NP>(a.A, d, a.N, part, in, A2);
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    A2[i] *= kLog2e;
    q[i] = 0.f;
  }
  float total[L::ITEMS][4] = {};
  sv.params(a.dt_bias, sBias);
  Pack<T, 4> rd[L::ITEMS], rz[L::ITEMS], ry[L::ITEMS];
  T rc[L::BCI];
  uint32_t od[L::ITEMS], oz[L::ITEMS], oy[L::ITEMS], oc[L::BCI];
#pragma unroll
  for (int k = 0; k < L::ITEMS; ++k) {
    od[k] = sv.offset(k, a.dt_row);
    oz[k] = sv.offset(k, a.z_row);
    oy[k] = sv.offset(k, a.D);
  }
#pragma unroll
  for (int k = 0; k < L::BCI; ++k) oc[k] = sv.bc_offset(k, a.c_row, a.N);
  auto fetch = [&](int at) {
    const int64_t t = sg.t0 + at;
    const int live = sg.len - at;
#pragma unroll
    for (int k = 0; k < L::ITEMS; ++k) {
      rd[k] = sv.load(a.dt, t, a.dt_row, od[k], k, live);
      ry[k] = sv.load(a.dy, t, a.D, oy[k], k, live);
      if (a.z != nullptr) rz[k] = sv.load(a.z, t, a.z_row, oz[k], k, live);
    }
#pragma unroll
    for (int k = 0; k < L::BCI; ++k) rc[k] = sv.load_bc(a.C, t, a.c_row, oc[k], k, a.N, live);
  };
  const int last = (sg.len - 1) / TT * TT;
  if (sg.len > 0) fetch(last);
  __syncthreads();
  for (int at = last; at >= 0 && sg.len > 0; at -= TT) {
    sv.renew();
    const int live = sg.len - at;
#pragma unroll
    for (int k = 0; k < L::ITEMS; ++k)
      if (sv.has(k)) {
        const bool ok = sv.token(k) < live;
        float bias[4];
        unpack(*reinterpret_cast<const float4*>(&sBias[sv.col(k)]), bias);
        float2* to = &sX[sv.token(k)][sv.col(k)];
        steps_of(rd[k], bias, a.softplus, ok, bias);
        float g[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) g[e] = ry[k].at(e);
        if (a.z != nullptr) gate_by(rz[k], g);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          total[k][e] += bias[e];
          to[e] = make_float2(bias[e], g[e]);
        }
      }
#pragma unroll
    for (int k = 0; k < L::BCI; ++k)
      if (sv.bc_has(k)) sC[sv.bc_token(k)][sv.bc_state(k)] = as_f(rc[k]);
    __syncthreads();
    if (at > 0) fetch(at - TT);
#pragma unroll
    for (int t = TT - 1; t >= 0; --t) {
      const float2 v = sX[t][chl];
      float cc[NPL];
      unpack(*reinterpret_cast<const float4*>(&sC[t][part * NPL]), cc);
#pragma unroll
      for (int i = 0; i < NPL; ++i) q[i] = exp2_hw(v.x * A2[i]) * fmaf(cc[i], v.y, q[i]);
    }
    __syncthreads();
  }
  const int64_t s = sg.first + sg.j;
  if (in) *reinterpret_cast<float4*>(a.seg_state + (s * a.D + d) * NP + part * NPL) = make_float4(q[0], q[1], q[2], q[3]);
  sum_dt<T, NP>(a, sv, total, reinterpret_cast<float*>(sX), s);
}

// Joins two values over the lanes that differ in bit D: a lane keeps the first value's sum where
// its bit is clear, the second's where it is set.
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
  if constexpr (D == 8) {
    const bool up = lane & 8;
    const float keep = up ? y : x, give = up ? x : y;
    return keep + dpp<kRor8>(give);
  }
}

// Backward of a segment, chunk by chunk from its end. From the saved state that enters a chunk its
// states and decays are formed again, the later half of the chunk first, into registers; then, in
// reverse, with dy' = dy silu(z),
//   r = C dy' + q,   q <- a r,   p = q h_{t-1},
//   dC += dy' h (summed over the group's channels),  dB += r dt x,  dA += dt p,
//   dx = dt sum_n r B + skip dy',   ddt = x sum_n r B + sum_n A p,   dz = dy y' silu'(z).
// Halves keep the states and decays of 8 tokens in registers rather than 16 (64 values a lane less), for
// the recurrence of the first 8 run twice: 166 us against 201 (B=2, T=2048, D=2048, N=16, bf16). Three waves
// a SIMD instead of two: 279 with halves (168 registers, 64 spilled), 153 against 145 with quarters, which
// fit but form the states of 12 tokens twice. The sums over channels are joined over the wave's lanes by
// merges (half the values move at each step), over the four waves in shared memory, and over
// channel tiles by a second kernel.
template <class T, int NP, bool GATE>
__global__ __launch_bounds__(256, 2) void sscan_bwd_kernel(ScanArgs a, int tiles) {
  typedef Lanes<NP> L;
  constexpr int HT = TT / 2;
  constexpr int LEFT = L::LPC >= 16 ? 2 : 1;  // of 8 values, what a lane ends with: the wave has 64 / LPC channels
  __shared__ float2 sX[TT][L::CH];          // dt, dt x
  __shared__ float sG[TT][L::CH];           // dy'; then sum_n r B
  __shared__ float sP[TT][L::CH];           // sum_n A p
  __shared__ float sY[GATE ? TT : 1][L::CH];  // y without skip and gate
  __shared__ float sB[TT][NP], sC[TT][NP];
  // a wave's dC (first NP), dB; behind them a place for the lanes that end with half sums
  __shared__ float sS[L::LPC <= 4 ? 8 : 4][TT][2 * NP];
  __shared__ float sBias[L::CH], sSkip[L::CH];
  const int bx = blockIdx.x % (a.G * tiles), grp = bx / tiles, tile = bx % tiles;
  const int c0 = tile * L::CH;
  const Segment sg = segment_at<false>(a, blockIdx.x / (a.G * tiles));
  Stage<T, NP> sv(a, grp, c0);
  const int tid = threadIdx.x, part = tid % L::LPC, chl = tid / L::LPC, lane = tid % 64, wave = tid / 64;
  const bool in = c0 + chl < sv.per;
  const int64_t d = (int64_t)grp * sv.per + c0 + chl;
  float A2[NPL], q[NPL], dA[NPL];
  load_states<NP>(a.A, d, a.N, part, in, A2);
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    A2[i] *= kLog2e;
    q[i] = dA[i] = 0.f;
  }
  if (a.dfinal != nullptr) load_states<NP>(a.dfinal, (int64_t)sg.n * a.D + d, a.N, part, in, q);
  if (in && a.split) {
    const int64_t count = segments_of(seq_end(a.sq, sg.n) - seq_begin(a.sq, sg.n), a.lseg);
    join_segments<NP>(a, sg.first_local + count - 1, -1, count - (int64_t)(sg.j + 1) * (a.seg / a.lseg), d, part, A2, q);
  }
  const int64_t chunk0 = sg.first_chunk + (int64_t)sg.j * (a.seg / TT);
  sv.params(a.dt_bias, sBias);
  sv.params(a.skip, sSkip);
  // where a lane's sum over channels goes: bit 5 dC or dB, bits 4 and 3 the state of its four
  float* to = &sS[L::LPC <= 4 && (lane & 7) >= L::LPC ? 4 + wave : wave][0]
                 [(lane >> 5) * NP + part * NPL + ((lane >> 4) & 1) * 2 + (LEFT == 1 ? (lane >> 3) & 1 : 0)];
  float dskip[L::ITEMS][4], dbias[L::ITEMS][4];
  Pack<T, 4> rx[L::ITEMS], rd[L::ITEMS], rz[L::ITEMS], ry[L::ITEMS];
  T rb[L::BCI], rc[L::BCI];
  float nh[NPL];
  uint32_t ox[L::ITEMS], od[L::ITEMS], oz[L::ITEMS], oy[L::ITEMS], ob[L::BCI], oc[L::BCI];
#pragma unroll
  for (int k = 0; k < L::ITEMS; ++k) {
    ox[k] = sv.offset(k, a.x_row);
    od[k] = sv.offset(k, a.dt_row);
    oz[k] = sv.offset(k, a.z_row);
    oy[k] = sv.offset(k, a.D);
#pragma unroll
    for (int e = 0; e < 4; ++e) dskip[k][e] = dbias[k][e] = 0.f;
  }
#pragma unroll
  for (int k = 0; k < L::BCI; ++k) {
    ob[k] = sv.bc_offset(k, a.b_row, a.N);
    oc[k] = sv.bc_offset(k, a.c_row, a.N);
  }
  auto fetch = [&](int at) {
    const int64_t t = sg.t0 + at;
    const int live = sg.len - at;
#pragma unroll
    for (int k = 0; k < L::ITEMS; ++k) {
      rx[k] = sv.load(a.x, t, a.x_row, ox[k], k, live);
      rd[k] = sv.load(a.dt, t, a.dt_row, od[k], k, live);
      ry[k] = sv.load(a.dy, t, a.D, oy[k], k, live);
      if (GATE) rz[k] = sv.load(a.z, t, a.z_row, oz[k], k, live);
    }
#pragma unroll
    for (int k = 0; k < L::BCI; ++k) {
      rb[k] = sv.load_bc(a.B, t, a.b_row, ob[k], k, a.N, live);
      rc[k] = sv.load_bc(a.C, t, a.c_row, oc[k], k, a.N, live);
    }
    load_states<NP>(a.states, (chunk0 + at / TT) * a.D + d, a.N, part, in, nh);
  };
  const int last = (sg.len - 1) / TT * TT;
  if (sg.len > 0) fetch(last);
  __syncthreads();
  for (int at = last; at >= 0 && sg.len > 0; at -= TT) {
    sv.renew();
    const int live = sg.len - at;
    Pack<T, 4> kx[L::ITEMS], kd[L::ITEMS], kz[L::ITEMS], ky[L::ITEMS];
    float h0[NPL], dAc[NPL];
#pragma unroll
    for (int k = 0; k < L::ITEMS; ++k) {
      if (L::ITEMS == 1) {
        kx[k] = rx[k];
        kd[k] = rd[k];
        kz[k] = rz[k];
        ky[k] = ry[k];
      }
      if (sv.has(k)) {
        const bool ok = sv.token(k) < live;
        float bias[4], g4[4];
        unpack(*reinterpret_cast<const float4*>(&sBias[sv.col(k)]), bias);
        float2* to = &sX[sv.token(k)][sv.col(k)];
        steps_of(rd[k], bias, a.softplus, ok, bias);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          g4[e] = ry[k].at(e);
          to[e] = make_float2(bias[e], bias[e] * rx[k].at(e));
        }
        if (GATE) gate_by(rz[k], g4);
        *reinterpret_cast<float4*>(&sG[sv.token(k)][sv.col(k)]) = make_float4(g4[0], g4[1], g4[2], g4[3]);
      }
    }
#pragma unroll
    for (int k = 0; k < L::BCI; ++k)
      if (sv.bc_has(k)) {
        sB[sv.bc_token(k)][sv.bc_state(k)] = as_f(rb[k]);
        sC[sv.bc_token(k)][sv.bc_state(k)] = as_f(rc[k]);
      }
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      h0[i] = nh[i];
      dAc[i] = 0.f;
    }
    __syncthreads();
    if (at > 0) fetch(at - TT);
    for (int half = 1; half >= 0; --half) {
      float hs[HT + 1][NPL], as[HT][NPL];
#pragma unroll
      for (int i = 0; i < NPL; ++i) hs[0][i] = h0[i];
      if (half == 1) {
#pragma unroll
        for (int t = 0; t < HT; ++t) {
          const float2 v = sX[t][chl];
          float bb[NPL];
          unpack(*reinterpret_cast<const float4*>(&sB[t][part * NPL]), bb);
#pragma unroll
          for (int i = 0; i < NPL; ++i) hs[0][i] = fmaf(exp2_hw(v.x * A2[i]), hs[0][i], v.y * bb[i]);
        }
      }
#pragma unroll
      for (int u = 0; u < HT; ++u) {
        const int t = half * HT + u;
        const float2 v = sX[t][chl];
        float bb[NPL];
        unpack(*reinterpret_cast<const float4*>(&sB[t][part * NPL]), bb);
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
          as[u][i] = exp2_hw(v.x * A2[i]);
          hs[u + 1][i] = fmaf(as[u][i], hs[u][i], v.y * bb[i]);
        }
        if (GATE) {
          float cc[NPL];
          unpack(*reinterpret_cast<const float4*>(&sC[t][part * NPL]), cc);
          float y = cc[0] * hs[u + 1][0];
#pragma unroll
          for (int i = 1; i < NPL; ++i) y = fmaf(cc[i], hs[u + 1][i], y);
          y = group_sum<L::LPC>(y);
          sY[t][chl] = y;  // the same from all lanes of the channel
        }
      }
      // The reverse walk loads B, C, dt and dt x again: without the opaque copies of the indexes the compiler
      // would keep them from the walk above, 80 registers a lane. A token's loads are issued one ahead.
      int rch = chl, rpart = part;
      asm volatile("" : "+v"(rch), "+v"(rpart));
      float2 nv = sX[half * HT + HT - 1][rch];
      float ng = sG[half * HT + HT - 1][rch];
      float4 nb = *reinterpret_cast<const float4*>(&sB[half * HT + HT - 1][rpart * NPL]);
      float4 nc = *reinterpret_cast<const float4*>(&sC[half * HT + HT - 1][rpart * NPL]);
#pragma unroll
      for (int u = HT - 1; u >= 0; --u) {
        const int t = half * HT + u;
        const float2 v = nv;
        const float g = ng;
        float bb[NPL], cc[NPL];
        unpack(nb, bb);
        unpack(nc, cc);
        if (u > 0) {
          nv = sX[t - 1][rch];
          ng = sG[t - 1][rch];
          nb = *reinterpret_cast<const float4*>(&sB[t - 1][rpart * NPL]);
          nc = *reinterpret_cast<const float4*>(&sC[t - 1][rpart * NPL]);
        }
        float s1 = 0.f, s2 = 0.f, val[8];
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
          const float r = fmaf(cc[i], g, q[i]);
          val[i] = g * hs[u + 1][i];
          val[4 + i] = r * v.y;
          s1 = fmaf(r, bb[i], s1);
          q[i] = as[u][i] * r;
          const float p = q[i] * hs[u][i];
          s2 = fmaf(p, A2[i], s2);
          dAc[i] = fmaf(p, v.x, dAc[i]);
        }
        s1 = group_sum<L::LPC>(s1);
        s2 = group_sum<L::LPC>(s2);
        sG[t][rch] = s1;  // only this channel's lanes, all of this wave, have read the place
        sP[t][rch] = s2;
        // val[0..3]: dC, val[4..7]: dB of this lane's four states; lanes of the wave with the same part
        // hold the other channels
        float m4[4], m2[2];
#pragma unroll
        for (int i = 0; i < 4; ++i) m4[i] = merge<32>(val[i], val[4 + i], lane);   // bit 5: dC or dB
#pragma unroll
        for (int i = 0; i < 2; ++i) m2[i] = merge<16>(m4[i], m4[2 + i], lane);     // bit 4: states 0, 1 or 2, 3
        if constexpr (LEFT == 2) {
          // LPC = 16: two values left, every lane's own
          to[t * 2 * NP] = m2[0];
          to[t * 2 * NP + 1] = m2[1];
        } else {
          float m = merge<8>(m2[0], m2[1], lane);                                  // bit 3: the one or the other
          if constexpr (L::LPC <= 2) m += dpp<kXor2>(m);
          if constexpr (L::LPC <= 4) m += dpp<kShl4>(m);                           // whole where bit 2 is clear
          to[t * 2 * NP] = m;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < NPL; ++i) dA[i] += dAc[i];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < L::ITEMS; ++k)
      if (sv.has(k)) {
        if (L::ITEMS > 1) {  // with two pieces a thread there are no registers to keep them over the walk
          const int64_t t = sg.t0 + at;
          kx[k] = sv.load(a.x, t, a.x_row, ox[k], k, live);
          kd[k] = sv.load(a.dt, t, a.dt_row, od[k], k, live);
          ky[k] = sv.load(a.dy, t, a.D, oy[k], k, live);
          if (GATE) kz[k] = sv.load(a.z, t, a.z_row, oz[k], k, live);
        }
        const int pt = sv.token(k), pc = sv.col(k);
        float vx[4], vd[4], vz[4], s1[4], s2[4], y[4], skip[4], bias[4];
        unpack(*reinterpret_cast<const float4*>(&sG[pt][pc]), s1);
        unpack(*reinterpret_cast<const float4*>(&sP[pt][pc]), s2);
        unpack(*reinterpret_cast<const float4*>(&sSkip[pc]), skip);
        unpack(*reinterpret_cast<const float4*>(&sBias[pc]), bias);
        if (GATE) unpack(*reinterpret_cast<const float4*>(&sY[pt][pc]), y);
        const bool ok = pt < live;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = kx[k].at(e);
          float g = ky[k].at(e);
          if (GATE) {
            const float z = kz[k].at(e), s = sigmoid(z);
            vz[e] = g * fmaf(skip[e], x, y[e]) * (s * fmaf(z, 1.f - s, 1.f));
            g *= z * s;
          }
          vx[e] = fmaf(sX[pt][pc + e].x, s1[e], skip[e] * g);
          vd[e] = fmaf(x, s1[e], s2[e] * kLn2);  // A2 holds A log2 e
          dskip[k][e] = fmaf(g, x, dskip[k][e]);
        }
        if (a.softplus) {
#pragma unroll
          for (int e = 0; e < 4; ++e) vd[e] *= sigmoid(kd[k].at(e) + bias[e]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) dbias[k][e] += ok ? vd[e] : 0.f;
        sv.store(a.dx, sg.t0 + at, a.D, oy[k], k, live, vx);
        sv.store(a.ddt, sg.t0 + at, a.D, oy[k], k, live, vd);
        if (a.dz != nullptr) sv.store(a.dz, sg.t0 + at, a.D, oy[k], k, live, vz);
      }
    for (int p = tid; p < TT * 2 * NP; p += 256) {
      const int pt = p / (2 * NP), v = p % (2 * NP);
      if (pt < live)
        a.part_bc[(((int64_t)tile * a.sq.total + sg.t0 + at + pt) * a.G + grp) * 2 * NP + v] =
            (sS[0][pt][v] + sS[1][pt][v]) + (sS[2][pt][v] + sS[3][pt][v]);
    }
    // no barrier: the next chunk's staging overwrites sX and sG only at the places that this thread itself
    // has just read, and sB and sC, which were last read before the barrier above
  }
  const int64_t s = sg.first + sg.j;
  if (a.dh0 != nullptr && sg.j == 0) store_states<NP>(a.dh0, (int64_t)sg.n * a.D + d, a.N, part, in, q);
  if (in) *reinterpret_cast<float4*>(a.part_a + (s * a.D + d) * NP + part * NPL) = make_float4(dA[0], dA[1], dA[2], dA[3]);
  // dskip and ddt_bias: the 16 threads that staged a channel join in shared memory
  for (int which = 0; which < 2; ++which) {
    __syncthreads();
#pragma unroll
    for (int k = 0; k < L::ITEMS; ++k)
      if (sv.has(k))
#pragma unroll
        for (int e = 0; e < 4; ++e) sG[sv.token(k)][sv.col(k) + e] = which == 0 ? dskip[k][e] : dbias[k][e];
    __syncthreads();
    if (tid < L::CH && c0 + tid < sv.per) {
      float sum = 0.f;
#pragma unroll
      for (int t = 0; t < TT; ++t) sum += sG[t][tid];
      a.part_d[(s * 2 + which) * a.D + (int64_t)grp * sv.per + c0 + tid] = sum;
    }
  }
}

// Joins the partial sums of a backward. The first bc_blocks workgroups: dB and dC from the channel tiles, four
// states a thread. The others: dA [D][N], dskip [D], ddt_bias [D] from the segments, 64 columns a
// workgroup with the segments dealt to 4 lanes a column. Fixed orders throughout.
template <class T, int NP>
__global__ __launch_bounds__(256) void sscan_sums_kernel(ScanArgs a, int tiles, int64_t bc_blocks) {
  __shared__ float sh[4][64];
  if ((int64_t)blockIdx.x < bc_blocks) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t rows = a.sq.total * a.G, row = i / (NP / 2);
    if (row >= rows) return;
    const int v = (int)(i % (NP / 2)) * 4, n = v % NP;  // the first NP of a row's 2 NP are dC
    const float4* p = reinterpret_cast<const float4*>(a.part_bc + row * 2 * NP + v);
    const int64_t step = rows * (NP / 2);
    float s[4] = {};
    for (int t = 0; t < tiles; t += 8) {
      float4 r[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (t + u < tiles) r[u] = p[(t + u) * step];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (t + u < tiles) {
          s[0] += r[u].x;
          s[1] += r[u].y;
          s[2] += r[u].z;
          s[3] += r[u].w;
        }
    }
    T* out = static_cast<T*>(v < NP ? a.dC : a.dB) + row * a.N + n;
    store_n<T, 4>(out, s, a.N - n, a.bcvec != 0);
    return;
  }
  const int tx = threadIdx.x % 64, ty = threadIdx.x / 64;
  const int64_t col = ((int64_t)blockIdx.x - bc_blocks) * 64 + tx, na = (int64_t)a.D * NP, cols = na + 2 * (int64_t)a.D;
  const float* p = col < na ? a.part_a + col : a.part_d + (col - na);
  const int64_t stride = col < na ? na : 2 * (int64_t)a.D;
  float s = 0.f;
  if (col < cols) {
#pragma unroll 4
    for (int64_t r = ty; r < a.nseg; r += 4) s += p[r * stride];
  }
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

// First segment, first local segment and first chunk of each packed sequence.
__global__ __launch_bounds__(1024) void sscan_tables_kernel(const int32_t* cu, int n, int seg, int lseg, int32_t* segoff,
                                                            int32_t* loff, int32_t* choff) {
  __shared__ int sh[3][1024];
  int base[3] = {0, 0, 0};
  int32_t* out[3] = {segoff, loff, choff};
  for (int i0 = 0; i0 < n; i0 += 1024) {
    const int i = i0 + threadIdx.x;
    const int len = i < n ? cu[i + 1] - cu[i] : 0;
    int mine[3] = {segments_of(len, seg), segments_of(len, lseg), chunks_of(len)};
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      if (i >= n) mine[k] = 0;
      sh[k][threadIdx.x] = mine[k];
    }
    __syncthreads();
    for (int step = 1; step < min(n - i0, 1024); step *= 2) {
      int add[3];
#pragma unroll
      for (int k = 0; k < 3; ++k) add[k] = (int)threadIdx.x >= step ? sh[k][threadIdx.x - step] : 0;
      __syncthreads();
#pragma unroll
      for (int k = 0; k < 3; ++k) sh[k][threadIdx.x] += add[k];
      __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      if (i < n) out[k][i] = base[k] + sh[k][threadIdx.x] - mine[k];
      base[k] += sh[k][min(n - i0, 1024) - 1];
    }
    __syncthreads();
  }
  if (threadIdx.x < 3) out[threadIdx.x][n] = base[threadIdx.x];
}

// One token: lanes as in the scan, the state read and written in place. A workgroup takes IT tiles of
// channels, all loaded before the slot is checked.
template <class T, int NP, int IT>
__global__ __launch_bounds__(256) void sscan_step_kernel(ScanStepArgs a, int tiles) {
  typedef Lanes<NP> L;
  const int per = a.D / a.G;
  const int grp = blockIdx.x / tiles, b = blockIdx.y;
  const int part = threadIdx.x % L::LPC;
  const int c0 = blockIdx.x % tiles * (L::CH * IT) + threadIdx.x / L::LPC;
  const int asked = a.slots != nullptr ? a.slots[b] : b;
  const bool held = asked >= 0 && asked < a.slots_n;
  const int64_t d0 = (int64_t)grp * per + c0, row0 = (int64_t)(held ? asked : 0) * a.D + d0;
  float h[IT][NPL], A[IT][NPL], x[IT], dt[IT], z[IT];
#pragma unroll
  for (int k = 0; k < IT; ++k) {
    const bool in = c0 + k * L::CH < per;
    const int64_t d = d0 + k * L::CH;
    if (a.N == NP) {
      unpack(in && held ? load_stream(a.state + (row0 + k * L::CH) * NP + part * NPL) : make_float4(0.f, 0.f, 0.f, 0.f), h[k]);
    } else {
      load_states<NP>(a.state, row0 + k * L::CH, a.N, part, in && held, h[k]);
    }
    load_states<NP>(a.A, d, a.N, part, in, A[k]);
    x[k] = in ? as_f(static_cast<const T*>(a.x)[b * a.x_row + d]) : 0.f;
    dt[k] = in ? as_f(static_cast<const T*>(a.dt)[b * a.dt_row + d]) + (a.dt_bias != nullptr ? a.dt_bias[d] : 0.f) : 0.f;
    z[k] = in && a.z != nullptr ? as_f(static_cast<const T*>(a.z)[b * a.z_row + d]) : 0.f;
  }
  float Bn[NPL], Cn[NPL];
  const T* Bm = static_cast<const T*>(a.Bm) + b * a.b_row + (int64_t)grp * a.N;
  const T* Cm = static_cast<const T*>(a.Cm) + b * a.c_row + (int64_t)grp * a.N;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int n = part * NPL + i;
    Bn[i] = n < a.N ? as_f(Bm[n]) : 0.f;
    Cn[i] = n < a.N ? as_f(Cm[n]) : 0.f;
  }
  const int slot = step_slot(a.slots, b, a.slots_n);
#pragma unroll
  for (int k = 0; k < IT; ++k) {
    if (c0 + k * L::CH < per) {
      const int64_t d = d0 + k * L::CH;
      T* y = static_cast<T*>(a.y) + (int64_t)b * a.D + d;
      if (slot < 0) {
        if (part == 0) *y = (T)(slot == -1 ? 0.f : __builtin_nanf(""));
      } else {
        const float step = a.softplus ? softplus(dt[k]) : dt[k];
        float out = 0.f;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
          h[k][i] = fmaf(exp2_hw(step * (A[k][i] * kLog2e)), h[k][i], step * x[k] * Bn[i]);
          out = fmaf(Cn[i], h[k][i], out);
        }
        if (a.N == NP)
          store_stream(a.state + (row0 + k * L::CH) * NP + part * NPL, make_float4(h[k][0], h[k][1], h[k][2], h[k][3]));
        else
          store_states<NP>(a.state, row0 + k * L::CH, a.N, part, true, h[k]);
        out = group_sum<L::LPC>(out);
        if (part == 0) {
          if (a.skip != nullptr) out = fmaf(a.skip[d], x[k], out);
          if (a.z != nullptr) out *= z[k] * sigmoid(z[k]);
          *y = (T)out;
        }
      }
    }
  }
}

template <class T, int NP>
hipError_t fwd_np(const ScanArgs& a, hipStream_t st) {
  const int tiles = scan_tiles(a.D, a.N, a.G);
  const dim3 grid((unsigned)(a.nseg * a.G * tiles));
  if (a.split) {
    const dim3 lgrid((unsigned)(a.nloc * a.G * tiles));
    hipLaunchKernelGGL((sscan_fwd_kernel<T, NP, false>), lgrid, dim3(256), 0, st, a, tiles);
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
    const dim3 lgrid((unsigned)(a.nloc * a.G * tiles));
    hipLaunchKernelGGL((sscan_bwd_local_kernel<T, NP>), lgrid, dim3(256), 0, st, a, tiles);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (a.z != nullptr)
    hipLaunchKernelGGL((sscan_bwd_kernel<T, NP, true>), grid, dim3(256), 0, st, a, tiles);
  else
    hipLaunchKernelGGL((sscan_bwd_kernel<T, NP, false>), grid, dim3(256), 0, st, a, tiles);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  const int64_t bc = (a.sq.total * a.G * (NP / 2) + 255) / 256, par = ((int64_t)a.D * (NP + 2) + 63) / 64;
  hipLaunchKernelGGL((sscan_sums_kernel<T, NP>), dim3((unsigned)(bc + par)), dim3(256), 0, st, a, tiles, bc);
  return hipGetLastError();
}

// Two tiles of channels a workgroup where that still gives two workgroups a CU, one otherwise (128 sequences,
// D = 4096, N = 16: 24.4, 19.5, 23.2 us with one, two, four).
template <class T, int NP>
hipError_t step_np(const ScanStepArgs& a, hipStream_t st) {
  const int ch = Lanes<NP>::CH, per = a.D / a.G, wide = (per + 2 * ch - 1) / (2 * ch);
  if ((int64_t)wide * a.G * a.B >= 512) {
    hipLaunchKernelGGL((sscan_step_kernel<T, NP, 2>), dim3(wide * a.G, a.B), dim3(256), 0, st, a, wide);
  } else {
    const int tiles = (per + ch - 1) / ch;
    hipLaunchKernelGGL((sscan_step_kernel<T, NP, 1>), dim3(tiles * a.G, a.B), dim3(256), 0, st, a, tiles);
  }
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

// Tokens of a segment and of a local one. A large call is cut into about four workgroups a CU (forward) or
// two (backward, whose registers allow no more), and where the longest sequence is at most two such
// segments not at all: the pass that a cut needs costs more than the fuller grid gives. A call that
// leaves the chip idle either way is cut for its latency: a chunk takes a workgroup alone 4 us (forward) or
// 8 (backward), a local segment joined on entry about 0.08, which balances at a seventh (a tenth) of the
// square root of the length in chunks; a ninth is taken for both. Local segments: shorter by up to four while that
// keeps the first pass within eight workgroups a CU and the joins few.
void scan_seg(const Seqs& s, int64_t longest, int D, int N, int G, bool bwd, int* seg, int* lseg) {
  const int64_t cols = (int64_t)G * scan_tiles(D, N, G), C = kScanChunk;
  const int64_t whole = longest > 0 ? (longest + C - 1) / C * C : C;
  const int64_t want = bwd ? 512 : 1024;
  int64_t least = 1;
  while (least * least * 36 * 36 < longest) ++least;  // ceil(sqrt(longest) / 36) chunks
  least *= C;
  int64_t len = ((s.total * cols + want - 1) / want + C - 1) / C * C;
  const bool small = len <= least;
  if (small) len = least;
  if (whole <= (small ? 4 : 2) * len) {
    *seg = *lseg = (int)whole;
    return;
  }
  int64_t r = 1;
  while (r < 4 && (s.total / len + s.n) * cols * r * 2 <= 2048 && len / (r * 2) >= least) r *= 2;
  len = (len + C * r - 1) / (C * r) * (C * r);
  *seg = (int)len;
  *lseg = (int)(len / r);
}

hipError_t launch_scan_tables(const Seqs& s, int seg, int lseg, int32_t* segoff, int32_t* loff, int32_t* choff,
                              hipStream_t st) {
  hipLaunchKernelGGL(sscan_tables_kernel, dim3(1), dim3(1024), 0, st, s.cu, s.n, seg, lseg, segoff, loff, choff);
  return hipGetLastError();
}

hipError_t launch_sscan_fwd(int dtype, const ScanArgs& a, hipStream_t st) { SSCAN_DISPATCH(fwd_np); }
hipError_t launch_sscan_bwd(int dtype, const ScanArgs& a, hipStream_t st) { SSCAN_DISPATCH(bwd_np); }
hipError_t launch_sscan_step(int dtype, const ScanStepArgs& a, hipStream_t st) { SSCAN_DISPATCH(step_np); }

}  // namespace kda
