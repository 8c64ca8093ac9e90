// Short causal convolution: forward, backward and single-token step.
//
// A thread owns VEC neighbouring channels and walks a run of tokens with the last W - 1 inputs in
// registers, so every input is loaded once per run plus W - 1 rows in front of it. The work is
// bound by memory: on B=4, T=4096, D=4096, W=4 in bf16 the forward moves its 268 MB in 54 us (5.0 TB/s; a large
// copy 5.2), the backward its 403 MB in 92 us (4.4 TB/s).
#include "layer_device.h"

namespace kda {

namespace {

// Tokens whose loads are issued together, while the ones before them are worked on. A multiple of
// every W (but 3), so that the windows need no moves between registers.
constexpr int kAhead = 4;
constexpr int kXcds = 8;

// Workgroups go to the eight XCDs in turn. Neighbouring runs of tokens share the rows between them, so
// each XCD, with its own L2, takes a stretch of neighbouring runs: n runs' blocks, this the i-th launched.
__device__ __forceinline__ int64_t stretch_of(int64_t i, int64_t n) {
  const int64_t q = n / kXcds, r = n % kXcds, x = i % kXcds;
  return x * q + min(x, r) + i / kXcds;
}

// A wave has one run of tokens: its tokens and sequences are scalars.
struct Cursor {
  int n;           // sequence of the current token
  int begin, end;  // its tokens
};

__device__ __forceinline__ Cursor cursor_at(const Seqs& s, int t) {
  Cursor c;
  c.n = seq_of(s, t);
  c.begin = (int)seq_begin(s, c.n);
  c.end = (int)seq_end(s, c.n);
  return c;
}
// The next sequence that has a token (the caller's token t is one).
__device__ __forceinline__ void advance(const Seqs& s, Cursor& c, int t) {
  while (t >= c.end) {
    ++c.n;
    c.begin = c.end;
    c.end = (int)seq_end(s, c.n);
  }
}

template <class T, int VEC>
__device__ __forceinline__ void load_row(const void* p, int64_t at, int valid, float (&out)[VEC]) {
  const auto v = load_n<T, VEC>(static_cast<const T*>(p) + at, valid, VEC > 1);
#pragma unroll
  for (int e = 0; e < VEC; ++e) out[e] = v.at(e);
}

// Row r of a sequence's history [h0 | tokens] (r < W - 1: h0), for `ch` and VEC - 1 channels behind it.
template <class T, int W, int VEC>
__device__ __forceinline__ void history_row(const ConvArgs& a, int n, int64_t begin, int64_t r, int ch, int valid,
                                            float (&out)[VEC]) {
  if (r >= W - 1) {
    load_row<T, VEC>(a.x, (begin + r - (W - 1)) * a.x_row + ch, valid, out);
  } else if (a.h0 != nullptr) {
    load_row<T, VEC>(a.h0, ((int64_t)n * (W - 1) + r) * a.D + ch, valid, out);
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) out[e] = 0.f;
  }
}

// The filters of VEC channels, VEC * W numbers in a row: 16 bytes a load where they are whole pieces of
// that and the array is aligned.
template <int W, int VEC>
__device__ __forceinline__ void load_filter(const float* weight, const float* bias, int wvec, int ch, float (&w)[W][VEC],
                                            float (&b)[VEC]) {
  float flat[VEC * W];
  if (VEC * W % 4 == 0 && wvec) {
    const float4* p = reinterpret_cast<const float4*>(weight + (int64_t)ch * W);
#pragma unroll
    for (int i = 0; i < VEC * W / 4; ++i) {
      const float4 v = p[i];
      flat[4 * i] = v.x;
      flat[4 * i + 1] = v.y;
      flat[4 * i + 2] = v.z;
      flat[4 * i + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC * W; ++i) flat[i] = weight[(int64_t)ch * W + i];
  }
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
#pragma unroll
    for (int j = 0; j < W; ++j) w[j][e] = flat[e * W + j];
    b[e] = bias != nullptr ? bias[ch + e] : 0.f;
  }
}

template <int W, int VEC>
__device__ __forceinline__ void push(float (&win)[W][VEC], const float (&x)[VEC]) {
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j) win[j][e] = win[j + 1][e];
    win[W - 1][e] = x[e];
  }
}
template <int W, int VEC>
__device__ __forceinline__ float tap_sum(const float (&w)[W][VEC], const float (&win)[W][VEC], float b, int e) {
  float u = b;
#pragma unroll
  for (int j = 0; j < W; ++j) u = fmaf(w[j][e], win[j][e], u);
  return u;
}

// Grid: (runs of tokens, then the sequences' final states) x channel blocks. Block: cx channel
// threads (whole waves) x 256 / cx runs.
template <class T, int W, int VEC>
__global__ __launch_bounds__(256) void conv_fwd_kernel(ConvArgs a, int cx, int64_t run_blocks) {
  const int tx = threadIdx.x % cx, rows = 256 / cx;
  const int ty = __builtin_amdgcn_readfirstlane(threadIdx.x / cx);
  const int64_t rb = blockIdx.x;
  const int ch = (blockIdx.y * cx + tx) * VEC;
  if (ch >= a.D) return;
  const int valid = VEC;  // D is a multiple of VEC
  if (rb >= run_blocks) {  // final state of `rows` sequences a block
    const int64_t n = (rb - run_blocks) * rows + ty;
    if (n >= a.sq.n) return;
    const int64_t begin = seq_begin(a.sq, (int)n), len = seq_end(a.sq, (int)n) - begin;
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
      float v[VEC];
      history_row<T, W, VEC>(a, (int)n, begin, len + i, ch, valid, v);
      store_n<T, VEC>(static_cast<T*>(a.final_state) + (n * (W - 1) + i) * a.D + ch, v, valid, VEC > 1);
    }
    return;
  }
  const int64_t run = stretch_of(rb, run_blocks) * rows + ty;
  if (run * a.tt >= a.sq.total) return;
  const int t0 = (int)(run * a.tt), t1 = (int)min((int64_t)t0 + a.tt, a.sq.total);
  const T* x = static_cast<const T*>(a.x);
  T* y = static_cast<T*>(a.y);
  Pack<T, VEC> next[kAhead];
  auto fetch = [&](int t) {
    if (t + kAhead <= t1) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) next[i] = load_n<T, VEC>(x + (t + i) * a.x_row + ch, valid, VEC > 1);
    }
  };
  fetch(t0);
  float w[W][VEC], b[VEC], win[W][VEC];  // win[j]: the input of tap j
  load_filter<W, VEC>(a.w, a.bias, a.wvec, ch, w, b);
  Cursor c = cursor_at(a.sq, t0);
#pragma unroll
  for (int j = 1; j < W; ++j) history_row<T, W, VEC>(a, c.n, c.begin, t0 - c.begin + j - 1, ch, valid, win[j]);
  auto token = [&](const Pack<T, VEC>& in, int t) {
    float v[VEC], out[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = in.at(e);
    push<W, VEC>(win, v);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float u = tap_sum<W, VEC>(w, win, b[e], e);
      out[e] = a.act ? u * sigmoid(u) : u;
    }
    store_n<T, VEC>(y + (int64_t)t * a.D + ch, out, valid, VEC > 1);
  };
  for (int t = t0; t < t1; t += kAhead) {
    if (t + kAhead <= min(t1, c.end)) {
      Pack<T, VEC> in[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) in[i] = next[i];
      fetch(t + kAhead);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) token(in[i], t + i);
    } else {  // a sequence ends in these tokens, or the run does
      fetch(t + kAhead);
#pragma unroll 1
      for (int s = t; s < min(t + kAhead, t1); ++s) {
        if (s >= c.end) {
          advance(a.sq, c, s);
#pragma unroll
          for (int j = 1; j < W; ++j) history_row<T, W, VEC>(a, c.n, c.begin, j - 1, ch, valid, win[j]);
        }
        token(load_n<T, VEC>(x + s * a.x_row + ch, valid, VEC > 1), s);
      }
    }
  }
}

// Backward of a run [t0, t1): du_t = dy_t act'(u_t) for its tokens and the W - 1 behind them (of
// their sequence), each added into the pending dx of the W tokens that it saw; dx of a token is
// whole once du of the token W - 1 behind it is in. The filter's gradient is summed over the run
// in registers, over the block's four runs in shared memory, and over blocks by a second kernel: one
// fixed order, no atomics.
template <class T, int W, int VEC>
__global__ __launch_bounds__(256) void conv_bwd_kernel(ConvArgs a, int64_t run_blocks) {
  __shared__ float sh[4][W + 1][64 * VEC];
  const int tx = threadIdx.x % 64;
  const int ty = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int64_t rb = blockIdx.x;
  const int ch = (blockIdx.y * 64 + tx) * VEC;
  const bool inside = ch < a.D;
  const int valid = VEC;  // D is a multiple of VEC
  const T* x = static_cast<const T*>(a.x);
  const T* dy = static_cast<const T*>(a.dy);
  float w[W][VEC], b[VEC];
  if (inside) load_filter<W, VEC>(a.w, a.bias, a.wvec, ch, w, b);
  if (rb >= run_blocks) {  // dh0 of four sequences a block: history rows 0 .. W - 2
    const int64_t n = (rb - run_blocks) * 4 + ty;
    if (n >= a.sq.n || !inside) return;
    const int64_t begin = seq_begin(a.sq, (int)n), len = seq_end(a.sq, (int)n) - begin;
    float acc[W - 1][VEC], win[W][VEC];
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) acc[i][e] = 0.f;
      history_row<T, W, VEC>(a, (int)n, begin, i, ch, valid, win[i + 1]);
      if (a.dfinal != nullptr && i >= len) load_row<T, VEC>(a.dfinal, (n * (W - 1) + i - len) * a.D + ch, valid, acc[i]);
    }
#pragma unroll
    for (int t = 0; t < W - 1; ++t) {
      if (t < len) {
        float in[VEC], g[VEC];
        load_row<T, VEC>(x, (begin + t) * a.x_row + ch, valid, in);
        load_row<T, VEC>(dy, (begin + t) * a.D + ch, valid, g);
        push<W, VEC>(win, in);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float u = tap_sum<W, VEC>(w, win, b[e], e);
          const float du = g[e] * (a.act ? dsilu(u) : 1.f);
#pragma unroll
          for (int j = 0; j < W; ++j)
            if (t + j < W - 1) acc[t + j][e] = fmaf(w[j][e], du, acc[t + j][e]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < W - 1; ++i)
      store_n<T, VEC>(static_cast<T*>(a.dh0) + (n * (W - 1) + i) * a.D + ch, acc[i], valid, VEC > 1);
    return;
  }
  const int64_t run = stretch_of(rb, run_blocks) * 4 + ty;
  float dw[W][VEC], db[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    db[e] = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) dw[j][e] = 0.f;
  }
  if (inside && run * a.tt < a.sq.total) {
    const int t0 = (int)(run * a.tt), t1 = (int)min((int64_t)t0 + a.tt, a.sq.total);
    const int t2 = (int)min((int64_t)t1 + W - 1, a.sq.total);
    T* dx = static_cast<T*>(a.dx) + ch;
    float win[W][VEC], pend[W][VEC];  // pend[m]: dx so far of the token W - 1 - m before the current one
    Pack<T, VEC> nx[kAhead], ng[kAhead];
    auto fetch = [&](int t) {
      if (t + kAhead <= t1) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          nx[i] = load_n<T, VEC>(x + (t + i) * a.x_row + ch, valid, VEC > 1);
          ng[i] = load_n<T, VEC>(dy + (int64_t)(t + i) * a.D + ch, valid, VEC > 1);
        }
      }
    };
    fetch(t0);
    Cursor c = cursor_at(a.sq, t0);
#pragma unroll
    for (int j = 1; j < W; ++j) history_row<T, W, VEC>(a, c.n, c.begin, t0 - c.begin + j - 1, ch, valid, win[j]);
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
      for (int e = 0; e < VEC; ++e) pend[j][e] = 0.f;
    const float zero[VEC] = {};
    // du of one token; what it adds to the pending dx from tap `from` on (the taps before it are h0's)
    auto token = [&](const Pack<T, VEC>& in, const Pack<T, VEC>& gin, int from, float mine) {
      float v[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[e] = in.at(e);
      push<W, VEC>(win, v);
      push<W, VEC>(pend, zero);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float u = tap_sum<W, VEC>(w, win, b[e], e);
        const float du = gin.at(e) * (a.act ? dsilu(u) : 1.f);
#pragma unroll
        for (int j = 0; j < W; ++j)
          if (j >= from) pend[j][e] = fmaf(w[j][e], du, pend[j][e]);
        const float own = mine == 1.f ? du : 0.f;
        db[e] += own;
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][e] = fmaf(own, win[j][e], dw[j][e]);
      }
    };
    for (int t = t0; t < t1 + W - 1; t += kAhead) {
      if (t - (W - 1) >= c.begin && t + kAhead + (W - 1) < c.end && t + kAhead <= t1) {
        // the run's own tokens, and those that get whole are clear of both ends of the sequence
        Pack<T, VEC> in[kAhead], g[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          in[i] = nx[i];
          g[i] = ng[i];
        }
        fetch(t + kAhead);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          token(in[i], g[i], 0, 1.f);
          if (t + i - (W - 1) >= t0) store_n<T, VEC>(dx + (int64_t)(t + i - (W - 1)) * a.D, pend[0], valid, VEC > 1);
        }
      } else {
        fetch(t + kAhead);
#pragma unroll 1
        for (int s = t; s < min(t + kAhead, t1 + W - 1); ++s) {
          const int done = s - (W - 1);  // the token whose dx is whole after s
          if (s < t2) {
            if (s >= c.end) {
              advance(a.sq, c, s);
#pragma unroll
              for (int j = 1; j < W; ++j) history_row<T, W, VEC>(a, c.n, c.begin, j - 1, ch, valid, win[j]);
            }
            token(load_n<T, VEC>(x + s * a.x_row + ch, valid, VEC > 1),
                  load_n<T, VEC>(dy + (int64_t)s * a.D + ch, valid, VEC > 1), W - 1 - (s - c.begin), s < t1 ? 1.f : 0.f);
          } else {
            push<W, VEC>(pend, zero);
          }
          if (done >= t0 && done < t1) {
            float v[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) v[e] = pend[0][e];
            if (a.dfinal != nullptr) {
              // rows len .. len + W - 2 of the history are the final state
              const Cursor f = done >= c.begin ? c : cursor_at(a.sq, done);
              const int r = (W - 1) - (f.end - done);
              if (r >= 0) {
                float d[VEC];
                load_row<T, VEC>(a.dfinal, ((int64_t)f.n * (W - 1) + r) * a.D + ch, valid, d);
#pragma unroll
                for (int e = 0; e < VEC; ++e) v[e] += d[e];
              }
            }
            store_n<T, VEC>(dx + (int64_t)done * a.D, v, valid, VEC > 1);
          }
        }
      }
    }
  }
  // one row of partial sums a block
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
#pragma unroll
    for (int j = 0; j < W; ++j) sh[ty][j][tx * VEC + e] = dw[j][e];
    sh[ty][W][tx * VEC + e] = db[e];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < (W + 1) * 64 * VEC; i += 256) {
    const int j = i / (64 * VEC), col = i % (64 * VEC);
    if ((int)blockIdx.y * 64 * VEC + col < a.D)
      a.part[((int64_t)rb * (W + 1) + j) * a.D + blockIdx.y * 64 * VEC + col] =
          (sh[0][j][col] + sh[1][j][col]) + (sh[2][j][col] + sh[3][j][col]);
  }
}

// dweight [D][W] and dbias [D] from [blocks][W + 1][D]; 64 columns a workgroup, the blocks' rows
// dealt to 16 lanes a column and joined in order.
template <int W>
__global__ __launch_bounds__(1024) void conv_filter_kernel(ConvArgs a, int64_t blocks) {
  __shared__ float sh[16][65];
  const int cols = (W + 1) * a.D;
  const int tx = threadIdx.x % 64, ty = threadIdx.x / 64;
  const int col = blockIdx.x * 64 + tx;
  float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
  if (col < cols) {
    int64_t r = ty;
    for (; r + 48 < blocks; r += 64) {
      s0 += a.part[r * cols + col];
      s1 += a.part[(r + 16) * cols + col];
      s2 += a.part[(r + 32) * cols + col];
      s3 += a.part[(r + 48) * cols + col];
    }
    for (; r < blocks; r += 16) s0 += a.part[r * cols + col];
  }
  sh[ty][tx] = (s0 + s1) + (s2 + s3);
  __syncthreads();
  if (ty == 0 && col < cols) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) s += sh[i][tx];
    const int j = col / a.D, ch = col % a.D;
    if (j < W) a.dw[(int64_t)ch * W + j] = s;
    else if (a.db != nullptr) a.db[ch] = s;
  }
}

template <class T, int W, int VEC>
__global__ __launch_bounds__(256) void conv_step_kernel(ConvStepArgs a) {
  const int row = blockIdx.y;
  const int ch = (blockIdx.x * 256 + threadIdx.x) * VEC;
  const int slot = step_slot(a.slots, row, a.slots_n);
  if (ch >= a.D) return;
  const int valid = VEC;  // D is a multiple of VEC
  T* y = static_cast<T*>(a.y) + (int64_t)row * a.D + ch;
  float out[VEC];
  if (slot < 0) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) out[e] = slot == -1 ? 0.f : __builtin_nanf("");
    store_n<T, VEC>(y, out, valid, VEC > 1);
    return;
  }
  T* st = static_cast<T*>(a.state) + (int64_t)slot * (W - 1) * a.D + ch;
  Pack<T, VEC> old[W - 1];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) old[j] = load_n<T, VEC>(st + (int64_t)j * a.D, valid, VEC > 1);
  const auto x = load_n<T, VEC>(static_cast<const T*>(a.x) + row * a.x_row + ch, valid, VEC > 1);
  float w[W][VEC], b[VEC];
  load_filter<W, VEC>(a.w, a.bias, a.wvec, ch, w, b);
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    float u = b[e];
#pragma unroll
    for (int j = 0; j < W; ++j) u = fmaf(w[j][e], (j < W - 1 ? old[j < W - 1 ? j : 0].at(e) : x.at(e)), u);
    out[e] = a.act ? u * sigmoid(u) : u;
  }
  store_n<T, VEC>(y, out, valid, VEC > 1);
#pragma unroll
  for (int j = 0; j < W - 1; ++j) {
    float v[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = j + 1 < W - 1 ? old[j + 1 < W - 1 ? j + 1 : 0].at(e) : x.at(e);
    store_n<T, VEC>(st + (int64_t)j * a.D, v, valid, VEC > 1);
  }
}

template <class T, int W>
hipError_t fwd_w(const ConvArgs& a, hipStream_t st) {
  const int cx = a.D <= 64 * a.vec ? 64 : 256, rows = 256 / cx;
  const int64_t runs = (a.sq.total + a.tt - 1) / a.tt, rb = (runs + rows - 1) / rows;
  const int64_t fb = a.final_state != nullptr ? (a.sq.n + rows - 1) / rows : 0;
  if (rb + fb == 0) return hipSuccess;
  const dim3 grid((unsigned)(rb + fb), (a.D + cx * a.vec - 1) / (cx * a.vec));
  if (a.vec == 4)
    hipLaunchKernelGGL((conv_fwd_kernel<T, W, 4>), grid, dim3(256), 0, st, a, cx, rb);
  else
    hipLaunchKernelGGL((conv_fwd_kernel<T, W, 1>), grid, dim3(256), 0, st, a, cx, rb);
  return hipGetLastError();
}

template <class T, int W>
hipError_t bwd_w(const ConvArgs& a, hipStream_t st) {
  // two channels a thread (96 registers, five waves a SIMD) take 92 us where four (two waves) take 97 on B=4,
  // T=4096, D=4096, W=4
  const int vec = a.vec > 1 ? 2 : 1;
  const int64_t rb = conv_row_blocks(a);
  const int64_t hb = a.dh0 != nullptr ? (a.sq.n + 3) / 4 : 0;
  const dim3 grid((unsigned)(rb + hb), (a.D + 64 * vec - 1) / (64 * vec));
  if (rb + hb > 0) {
    if (vec == 2)
      hipLaunchKernelGGL((conv_bwd_kernel<T, W, 2>), grid, dim3(256), 0, st, a, rb);
    else
      hipLaunchKernelGGL((conv_bwd_kernel<T, W, 1>), grid, dim3(256), 0, st, a, rb);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((conv_filter_kernel<W>), dim3(((W + 1) * a.D + 63) / 64), dim3(1024), 0, st, a, rb);
  return hipGetLastError();
}

template <class T, int W>
hipError_t step_w(const ConvStepArgs& a, hipStream_t st) {
  const void* p[3] = {a.x, a.state, a.y};
  const int vec = conv_vec(sizeof(T) == 4 ? KDA_F32 : KDA_BF16, a.D, a.x_row, p, 3) > 1 ? 4 : 1;
  const dim3 grid((a.D + 256 * vec - 1) / (256 * vec), a.B);
  if (vec == 4)
    hipLaunchKernelGGL((conv_step_kernel<T, W, 4>), grid, dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL((conv_step_kernel<T, W, 1>), grid, dim3(256), 0, st, a);
  return hipGetLastError();
}

#define CONV_DISPATCH(FN, A)                                             \
  do {                                                                   \
    if (dtype == KDA_F32) {                                              \
      if ((A).W == 2) return FN<float, 2>(A, st);                        \
      if ((A).W == 3) return FN<float, 3>(A, st);                        \
      return FN<float, 4>(A, st);                                        \
    }                                                                    \
    if ((A).W == 2) return FN<bf16, 2>(A, st);                           \
    if ((A).W == 3) return FN<bf16, 3>(A, st);                           \
    return FN<bf16, 4>(A, st);                                           \
  } while (0)

}  // namespace

// Channels of a thread: four where every row starts on a multiple of them, single ones otherwise.
// (Eight bf16 channels, 16 bytes a load, take 56 us where four take 54 on B=4, T=4096, D=4096, W=4: filter,
// window and rows ahead of eight channels leave fewer waves a SIMD.)
int conv_vec(int dtype, int D, int64_t x_row, const void* const* ptrs, int np) {
  const int es = dtype == KDA_F32 ? 4 : 2;
  bool ok = D % 4 == 0 && x_row % 4 == 0;
  for (int i = 0; i < np; ++i) ok = ok && reinterpret_cast<uintptr_t>(ptrs[i]) % (4 * es) == 0;
  return ok ? 4 : 1;
}

// Tokens of a run: as many as leave about 2048 waves, from 8 to 64 (a longer run reads its W - 1
// rows in front less often, a shorter one gives more waves to a small call). 64 against 32 on
// B=4, T=4096, D=4096: forward 54 against 60 us, backward 92 against 98.
int conv_tile(int64_t total, int D, int vec) {
  const int64_t cols = (D + vec - 1) / vec;
  int tt = 64;
  while (tt > 8 && (total + tt - 1) / tt * cols < 2048 * 64) tt /= 2;
  return tt;
}

int64_t conv_row_blocks(const ConvArgs& a) { return ((a.sq.total + a.tt - 1) / a.tt + 3) / 4; }

hipError_t launch_conv_fwd(int dtype, const ConvArgs& a, hipStream_t st) { CONV_DISPATCH(fwd_w, a); }
hipError_t launch_conv_bwd(int dtype, const ConvArgs& a, hipStream_t st) { CONV_DISPATCH(bwd_w, a); }
hipError_t launch_conv_step(int dtype, const ConvStepArgs& a, hipStream_t st) { CONV_DISPATCH(step_w, a); }

}  // namespace kda
