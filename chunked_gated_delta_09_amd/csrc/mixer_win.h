// Attention with a sliding window and first tokens that stay visible: forward and backward over whole sequences.
//
// Token i sees j <= i where i - j < window or j < sinks. A workgroup takes a run of queries of one head and goes over the tiles
// of keys that they see: those of the first tokens, then the window's, with the running maximum and sum of a softmax.
// Scores are formed transposed, S^T = K Q^T: a lane then holds scores of one query (column l % 16), its maximum, sum and
// rescaling are the lane's own numbers, and P^T is an operand of O^T += V^T P^T as it stands (stacked order), with V^T read
// transposed from shared memory. Backward, with delta_i = do_i.o_i:
//   P_ij = exp(scale q_i.k_j - lse_i),  dS_ij = P_ij (do_i.v_j - delta_i),
//   dq_i = scale sum_j dS_ij k_j  (runs of queries over tiles of keys),  dk_j = scale sum_i dS_ij q_i,  dv_j = sum_i P_ij do_i  (runs of keys
// over tiles of queries, all heads of the key head one after the other, so that gradients of shared heads are sums
// in registers). Scores are formed twice in the backward; that needs no sums across workgroups. The first tokens' keys
// are seen by all queries behind the window too: those are dealt to workgroups of their own in parts, whose sums
// are added in order.
//
// Scores, statistics, P before its product, and all sums are fp32. P and dS are rounded to the type as operands (2^-9
// relative each for bf16, as their outputs' own rounding).
//
// Measured, bf16: forward of a prompt of 16384 tokens, 16 heads of 128 channels, window 4096 606 us (790 TFLOP/s); training B=2, T=4096, 32
// heads over 8, window 1024: forward 208, dq 272, dk and dv 378, first tokens 35 us. The vector unit (a score's scaling, exponential, maximum
// and sum) and the matrix unit have work for about a third of the time each, shared memory for 15 to 30 %; two waves a SIMD overlap them in part.
#pragma once

#include <type_traits>

#include "mixer_device.h"

namespace kda {

template <class T>
struct WinTile {
  static constexpr int KB = sizeof(T) == 2 ? 64 : 32;  // rows of a tile in shared memory
};

// Tiles of keys that a run of queries goes over: `sinks` of them from the first key, then `lo` to `hi`.
struct KeyTiles {
  int sinks, lo, count;
  __device__ __forceinline__ int at(int i) const { return i < sinks ? i : lo + i - sinks; }
};
__device__ __forceinline__ KeyTiles key_tiles(const WinArgs& a, int q0, int q1, int kb) {
  KeyTiles t;
  t.lo = max(0, q0 - a.window + 1) / kb;
  t.sinks = min((a.sinks + kb - 1) / kb, t.lo);
  t.count = t.sinks + q1 / kb - t.lo + 1;
  return t;
}

__device__ __forceinline__ bool sees(const WinArgs& a, int i, int j) { return j <= i && (i - j < a.window || j < a.sinks); }

// A key's values (or a query's, in the sums over queries) reach only what sees it, whatever they hold: a mask makes its weight
// zero, but zero times an infinity is NaN. So where a result is not finite, the workgroup forms its results once more, and leaves
// what is not finite out of the products of partly masked tiles; this adds it where it is seen. (A look at the results
// costs nothing beside one at the values of all such tiles.)
template <class T, int DP, int N, class Sees>
__device__ __forceinline__ void add_not_finite(const T* tile, int rows, f32x4 (&acc)[DP / 16][N], Sees sees) {
  typedef Tile<T, DP> L;
  int tid = threadIdx.x;
  asm volatile("" : "+v"(tid));  // nothing of this is held through the loops around it
  const int g4 = tid % 64 / 16;
#pragma unroll 1
  for (int r = 0; r < rows; ++r)
#pragma unroll
    for (int d = 0; d < DP / 16; ++d) {
      const int c = d * 16 + 4 * g4, per = 16 / (int)sizeof(T);
      const auto x = load_n<T, 4>(tile + L::block(r, c / per) + c % per, 4, true);
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (!(fabsf(x.at(e)) < INFINITY) && sees(n, r)) acc[d][n][e] += x.at(e);
    }
}
// Whether a wave's 32 rows hold something that is not finite.
template <class T, int DP>
__device__ __forceinline__ bool rows_not_finite(const T* tile) {
  typedef Tile<T, DP> L;
  constexpr int EV = 16 / (int)sizeof(T), PER = DP / EV;
  float sum = 0.f;
  int tid = threadIdx.x;
  asm volatile("" : "+v"(tid));  // as above
#pragma unroll 1
  for (int b = tid % 64; b < 32 * PER; b += 64) {
    const auto x = load_n<T, EV>(tile + L::block(b / PER, b % PER), EV, true);
#pragma unroll
    for (int e = 0; e < EV; ++e) sum = fmaf(x.at(e), 0.f, sum);
  }
  return __any(!(sum == 0.f));
}
__device__ __forceinline__ bool any_not_finite(float sum) {
  return __builtin_amdgcn_readfirstlane(__syncthreads_or(!(sum == 0.f))) != 0;
}

template <class T, int DP, int QT, int MODE>
__global__ __launch_bounds__(256, sizeof(T) == 2 && DP <= 128 ? 2 : 1) void win_fwd_kernel(WinArgs a) {
  constexpr int KB = WinTile<T>::KB, KT = KB / 16, DS = DP / 32, DT = DP / 16, QB = 64 * QT;
  constexpr bool VEC = MODE != kOdd, DIRECT = MODE == kDirect;
  typedef Tile<T, DP> L;
  typedef Feed<T, KB, DP, MODE> F;
  __shared__ __align__(16) T sk[F::BUFFERS * F::SIZE], sv[F::BUFFERS * F::SIZE];
  const int lane = threadIdx.x % 64, l16 = lane % 16, g4 = lane / 16;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int64_t id = xcd_order(blockIdx.x, gridDim.x);
  const int h = (int)(id / a.blocks), blk = (int)(id % a.blocks), hk = h / (a.H / a.HK);
  const Span sp = find_span(a.sq, QB, blk);
  const int q0 = sp.s * QB;
  if (q0 >= sp.len) return;  // a sequence without tokens
  const int q1 = min(q0 + QB, sp.len) - 1, qa = q0 + wave * 16 * QT;
  const T* k = static_cast<const T*>(a.k) + sp.seq0 * a.k_row + (int64_t)hk * a.D;
  const T* v = static_cast<const T*>(a.v) + sp.seq0 * a.v_row + (int64_t)hk * a.D;

  Frag<T> qf[QT][DS];
#pragma unroll
  for (int qt = 0; qt < QT; ++qt) {
    const int i = qa + qt * 16 + l16;
    const T* q = static_cast<const T*>(a.q) + (sp.seq0 + i) * a.q_row + (int64_t)h * a.D;
#pragma unroll
    for (int s = 0; s < DS; ++s) {
      qf[qt][s] = row_global<VEC>(q, s * 32, i < sp.len ? a.D : 0);
      if (a.scale < 0.f) qf[qt][s] = -qf[qt][s];  // the scale is at least zero below: it keeps the order of scores
    }
  }
  f32x4 o[DT][QT];
  float m[QT], l[QT];
  const float scale2 = fmaxf(fabsf(a.scale) * kLog2e, 1e-30f);  // not zero: a masked score times it stays -infinity
  const KeyTiles kt = key_tiles(a, q0, q1, KB);
  auto pass = [&](auto again) __attribute__((always_inline)) {
    F fk, fv;
    auto fetch = [&](int t, int b) {
      const int64_t at = (int64_t)t * KB;
      fk.fetch(k + at * a.k_row, (int)a.k_row, sp.len - t * KB, a.D, sk + b * F::SIZE);
      fv.fetch(v + at * a.v_row, (int)a.v_row, sp.len - t * KB, a.D, sv + b * F::SIZE);
    };
#pragma unroll
    for (int qt = 0; qt < QT; ++qt) {
      m[qt] = -INFINITY;
      l[qt] = 0.f;
#pragma unroll
      for (int d = 0; d < DT; ++d) o[d][qt] = zero4();
    }
    fetch(kt.at(0), 0);
    for (int it = 0; it < kt.count; ++it) {
      const int ka = kt.at(it) * KB, kb = ka + KB - 1, qb = qa + 16 * QT - 1;
      const int buf = DIRECT ? it % 2 : 0;
      const T *tk = sk + buf * F::SIZE, *tv = sv + buf * F::SIZE;
      if constexpr (DIRECT) loads_done();
      __syncthreads();
      if constexpr (!DIRECT) {
        fk.store(sk);
        fv.store(sv);
        __syncthreads();
      }
      if (it + 1 < kt.count) fetch(kt.at(it + 1), 1 - buf);
      if (ka > qb || !(qa - kb < a.window || ka < a.sinks)) continue;  // nothing for this wave's queries
      const bool full = kb <= qa && (qb - ka < a.window || kb < a.sinks);
      f32x4 s[KT][QT];
#pragma unroll
      for (int t = 0; t < KT; ++t) {
#pragma unroll
        for (int qt = 0; qt < QT; ++qt) s[t][qt] = zero4();
#pragma unroll
        for (int ds = 0; ds < DS; ++ds) {
          const Frag<T> kf = L::row(tk, t * 16, ds * 32);
#pragma unroll
          for (int qt = 0; qt < QT; ++qt) s[t][qt] = mma(kf, qf[qt][ds], s[t][qt]);
        }
      }
      if constexpr (sizeof(T) == 2 && !again.value) alternate<KT, DS, DS * QT>();  // 623 -> 614 us, prompt of 16384 tokens
#pragma unroll
      for (int qt = 0; qt < QT; ++qt) {
        const int i = qa + qt * 16 + l16;
        if (!full) {
#pragma unroll
          for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (!sees(a, i, ka + t * 16 + 4 * g4 + e)) s[t][qt][e] = -INFINITY;
        }
        float high = s[0][qt][0];
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) high = fmaxf(high, s[t][qt][e]);
        high = fmaxf(high, __shfl_xor(high, 16));
        high = fmaxf(high, __shfl_xor(high, 32));
        const float top = fmaxf(m[qt], high == -INFINITY ? high : high * scale2);
        const float base = top == -INFINITY ? 0.f : top;  // a row that has seen nothing yet
        if (__any(top > m[qt])) {  // else nothing is rescaled
          const float down = exp2_hw(m[qt] - base);
          m[qt] = top;
          l[qt] *= down;
#pragma unroll
          for (int d = 0; d < DT; ++d) o[d][qt] *= down;
        }
        float sum = 0.f;
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float p = exp2_hw(fmaf(s[t][qt][e], scale2, -base));
            s[t][qt][e] = p;
            sum += p;
          }
        l[qt] += sum;
      }
      auto product = [&](auto finite) __attribute__((always_inline)) {
#pragma unroll
        for (int js = 0; js < KB / 32; ++js) {
          Frag<T> pf[QT];
#pragma unroll
          for (int qt = 0; qt < QT; ++qt) pf[qt] = to_frag<T>(stack(s[2 * js][qt], s[2 * js + 1][qt]));
#pragma unroll
          for (int d = 0; d < DT; ++d) {
            Frag<T> vf = L::col(tv, js * 32, d * 16);
            if constexpr (finite.value) {
              vf = finite_only(vf);
              __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int qt = 0; qt < QT; ++qt) o[d][qt] = mma(vf, pf[qt], o[d][qt]);
          }
        }
      };
      if (again.value && !full) {
        product(again);
        add_not_finite<T, DP>(tv, KB, o, [&](int qt, int r) { return sees(a, qa + qt * 16 + l16, ka + r); });
      } else {
        product(std::false_type());
      }
    }
    float sum = 0.f;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int qt = 0; qt < QT; ++qt) sum = times_zero(o[d][qt], sum);
    return !again.value && any_not_finite(sum);
  };
  if (pass(std::false_type())) pass(std::true_type());
#pragma unroll
  for (int qt = 0; qt < QT; ++qt) {
    const int i = qa + qt * 16 + l16;
    const float sum = add_xor32(add_xor16(l[qt])), inv = 1.f / sum;
    if (i >= sp.len) continue;
    const int64_t row = (sp.seq0 + i) * a.H + h;
    if (a.lse != nullptr && g4 == 0) a.lse[row] = (m[qt] + __builtin_amdgcn_logf(sum)) * kLn2;
    T* out = static_cast<T*>(a.o) + row * a.D;
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      const int c = d * 16 + 4 * g4;
      const float x[4] = {o[d][qt][0] * inv, o[d][qt][1] * inv, o[d][qt][2] * inv, o[d][qt][3] * inv};
      if (c < a.D) store_n<T, 4>(out + c, x, a.D - c, VEC);
    }
  }
}

template <class T, int DP, int QT, int MODE>
__global__ __launch_bounds__(256, sizeof(T) == 2 && DP <= 128 ? 2 : 1) void win_dq_kernel(WinArgs a) {
  constexpr int KB = WinTile<T>::KB, KT = KB / 16, DS = DP / 32, DT = DP / 16, QB = 64 * QT;
  constexpr bool VEC = MODE != kOdd, DIRECT = MODE == kDirect;
  typedef Tile<T, DP> L;
  typedef Feed<T, KB, DP, MODE> F;
  __shared__ __align__(16) T sk[F::BUFFERS * F::SIZE], sv[F::BUFFERS * F::SIZE];
  const int lane = threadIdx.x % 64, l16 = lane % 16, g4 = lane / 16;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int64_t id = xcd_order(blockIdx.x, gridDim.x);
  const int h = (int)(id / a.blocks), blk = (int)(id % a.blocks), hk = h / (a.H / a.HK);
  const Span sp = find_span(a.sq, QB, blk);
  const int q0 = sp.s * QB;
  if (q0 >= sp.len) return;
  const int q1 = min(q0 + QB, sp.len) - 1, qa = q0 + wave * 16 * QT;
  const T* k = static_cast<const T*>(a.k) + sp.seq0 * a.k_row + (int64_t)hk * a.D;
  const T* v = static_cast<const T*>(a.v) + sp.seq0 * a.v_row + (int64_t)hk * a.D;

  Frag<T> qf[QT][DS], df[QT][DS];
  float lse2[QT], delta[QT];
#pragma unroll
  for (int qt = 0; qt < QT; ++qt) {
    const int i = qa + qt * 16 + l16;
    const bool in = i < sp.len;
    const int64_t row = (sp.seq0 + i) * a.H + h;
    const T* q = static_cast<const T*>(a.q) + (sp.seq0 + i) * a.q_row + (int64_t)h * a.D;
    const T* d = static_cast<const T*>(a.dout) + row * a.D;
    const T* o = static_cast<const T*>(a.out) + row * a.D;
    lse2[qt] = in ? a.lse_in[row] * kLog2e : INFINITY;
    float sum = 0.f;
#pragma unroll
    for (int s = 0; s < DS; ++s) {
      qf[qt][s] = row_global<VEC>(q, s * 32, in ? a.D : 0);
      df[qt][s] = row_global<VEC>(d, s * 32, in ? a.D : 0);
      const f32x8 x = to_f32<T>(df[qt][s]), y = to_f32<T>(row_global<VEC>(o, s * 32, in ? a.D : 0));
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = fmaf(x[e], y[e], sum);
    }
    delta[qt] = add_xor32(add_xor16(sum));
    if (in && g4 == 0) a.delta[row] = delta[qt];
  }
  f32x4 dq[DT][QT];
  const float scale2 = a.scale * kLog2e;
  const KeyTiles kt = key_tiles(a, q0, q1, KB);
  auto pass = [&](auto again) __attribute__((always_inline)) {
    F fk, fv;
    auto fetch = [&](int t, int b) {
      const int64_t at = (int64_t)t * KB;
      fk.fetch(k + at * a.k_row, (int)a.k_row, sp.len - t * KB, a.D, sk + b * F::SIZE);
      fv.fetch(v + at * a.v_row, (int)a.v_row, sp.len - t * KB, a.D, sv + b * F::SIZE);
    };
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int qt = 0; qt < QT; ++qt) dq[d][qt] = zero4();
    fetch(kt.at(0), 0);
    for (int it = 0; it < kt.count; ++it) {
      const int ka = kt.at(it) * KB, kb = ka + KB - 1, qb = qa + 16 * QT - 1;
      const int buf = DIRECT ? it % 2 : 0;
      const T *tk = sk + buf * F::SIZE, *tv = sv + buf * F::SIZE;
      if constexpr (DIRECT) loads_done();
      __syncthreads();
      if constexpr (!DIRECT) {
        fk.store(sk);
        fv.store(sv);
        __syncthreads();
      }
      if (it + 1 < kt.count) fetch(kt.at(it + 1), 1 - buf);
      if (ka > qb || !(qa - kb < a.window || ka < a.sinks)) continue;
      const bool full = kb <= qa && (qb - ka < a.window || kb < a.sinks);
#pragma unroll
      for (int js = 0; js < KB / 32; ++js) {
        f32x4 s[2][QT], dp[2][QT];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int row = (js * 2 + t) * 16;
#pragma unroll
          for (int qt = 0; qt < QT; ++qt) s[t][qt] = dp[t][qt] = zero4();
#pragma unroll
          for (int ds = 0; ds < DS; ++ds) {
            const Frag<T> kf = L::row(tk, row, ds * 32), vf = L::row(tv, row, ds * 32);
#pragma unroll
            for (int qt = 0; qt < QT; ++qt) {
              s[t][qt] = mma(kf, qf[qt][ds], s[t][qt]);
              dp[t][qt] = mma(vf, df[qt][ds], dp[t][qt]);
            }
          }
#pragma unroll
          for (int qt = 0; qt < QT; ++qt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int i = qa + qt * 16 + l16, j = ka + (js * 2 + t) * 16 + 4 * g4 + e;
              float p = exp2_hw(fmaf(s[t][qt][e], scale2, -lse2[qt]));
              if (!full && !sees(a, i, j)) p = 0.f;
              s[t][qt][e] = p == 0.f ? 0.f : p * (dp[t][qt][e] - delta[qt]);
            }
        }
        Frag<T> sf[QT];
#pragma unroll
        for (int qt = 0; qt < QT; ++qt) sf[qt] = to_frag<T>(stack(s[0][qt], s[1][qt]));
        auto product = [&](auto finite) __attribute__((always_inline)) {
#pragma unroll
          for (int d = 0; d < DT; ++d) {
            Frag<T> kf = L::col(tk, js * 32, d * 16);
            if constexpr (finite.value) {
              kf = finite_only(kf);
              __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int qt = 0; qt < QT; ++qt) dq[d][qt] = mma(kf, sf[qt], dq[d][qt]);
          }
        };
        if (again.value && !full) product(again);
        else product(std::false_type());
      }
      if (again.value && !full) add_not_finite<T, DP>(tk, KB, dq, [&](int qt, int r) { return sees(a, qa + qt * 16 + l16, ka + r); });
    }
    float sum = 0.f;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int qt = 0; qt < QT; ++qt) sum = times_zero(dq[d][qt], sum);
    return !again.value && any_not_finite(sum);
  };
  if (pass(std::false_type())) pass(std::true_type());
#pragma unroll
  for (int qt = 0; qt < QT; ++qt) {
    const int i = qa + qt * 16 + l16;
    if (i >= sp.len) continue;
    T* out = static_cast<T*>(a.dq) + ((sp.seq0 + i) * a.H + h) * a.D;
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      const int c = d * 16 + 4 * g4;
      const float x[4] = {dq[d][qt][0] * a.scale, dq[d][qt][1] * a.scale, dq[d][qt][2] * a.scale, dq[d][qt][3] * a.scale};
      if (c < a.D) store_n<T, 4>(out + c, x, a.D - c, VEC);
    }
  }
}

// A run of keys over the tiles of queries that see them through the window.
template <class T, int DP, int KT, int MODE>
__global__ __launch_bounds__(256, sizeof(T) == 2 && DP <= 128 ? 2 : 1) void win_dkv_kernel(WinArgs a) {
  constexpr int QB = WinTile<T>::KB, DS = DP / 32, DT = DP / 16, KB = 64 * KT;
  constexpr bool VEC = MODE != kOdd, DIRECT = MODE == kDirect;
  typedef Tile<T, DP> L;
  typedef Feed<T, QB, DP, MODE> F;
  __shared__ __align__(16) T sq[F::BUFFERS * F::SIZE], sd[F::BUFFERS * F::SIZE];
  __shared__ __align__(16) float sl[F::BUFFERS][QB], se[F::BUFFERS][QB];
  const int tid = threadIdx.x, lane = tid % 64, l16 = lane % 16, g4 = lane / 16;
  const int wave = __builtin_amdgcn_readfirstlane(tid / 64);
  const int64_t id = xcd_order(blockIdx.x, gridDim.x);
  const int rep = a.H / a.HK;
  const int hk = (int)(id / a.blocks);
  const Span sp = find_span(a.sq, KB, (int)(id % a.blocks));
  const int k0 = sp.s * KB;
  if (k0 >= sp.len) return;
  const int qlo = k0, qhi = (int)min((int64_t)sp.len, (int64_t)min(k0 + KB, sp.len) - 1 + a.window) - 1;
  const int ka = k0 + wave * 16 * KT, kb = ka + 16 * KT - 1;
  Frag<T> kf[KT][DS], vf[KT][DS];
#pragma unroll
  for (int kt = 0; kt < KT; ++kt) {
    const int j = ka + kt * 16 + l16;
    const T* k = static_cast<const T*>(a.k) + (sp.seq0 + j) * a.k_row + (int64_t)hk * a.D;
    const T* v = static_cast<const T*>(a.v) + (sp.seq0 + j) * a.v_row + (int64_t)hk * a.D;
#pragma unroll
    for (int s = 0; s < DS; ++s) {
      kf[kt][s] = row_global<VEC>(k, s * 32, j < sp.len ? a.D : 0);
      vf[kt][s] = row_global<VEC>(v, s * 32, j < sp.len ? a.D : 0);
    }
  }
  f32x4 dk[DT][KT], dv[DT][KT];
  const float scale2 = a.scale * kLog2e;
  const int t0 = qlo / QB, tn = qhi / QB - t0 + 1;
  auto pass = [&](auto again) __attribute__((always_inline)) {
    F fq, fd;
    float fl = 0.f, fe = 0.f;
    auto fetch = [&](int i, int b) {
      const int h = hk * rep + i / tn, t = t0 + i % tn, rows = sp.len - t * QB;
      const int64_t at = sp.seq0 + (int64_t)t * QB;
      fq.fetch(static_cast<const T*>(a.q) + at * a.q_row + (int64_t)h * a.D, (int)a.q_row, rows, a.D, sq + b * F::SIZE);
      fd.fetch(static_cast<const T*>(a.dout) + (at * a.H + h) * a.D, a.H * a.D, rows, a.D, sd + b * F::SIZE);
      if (tid < QB) {
        fl = tid < rows ? a.lse_in[(at + tid) * a.H + h] * kLog2e : INFINITY;
        fe = tid < rows ? a.delta[(at + tid) * a.H + h] : 0.f;
      }
    };
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) dk[d][kt] = dv[d][kt] = zero4();
    fetch(0, 0);
    for (int i = 0; i < rep * tn; ++i) {
      const int qa = (t0 + i % tn) * QB, qb = qa + QB - 1;
      const int buf = DIRECT ? i % 2 : 0;
      const T *tq = sq + buf * F::SIZE, *td = sd + buf * F::SIZE;
      if constexpr (!DIRECT) __syncthreads();
      fq.store(sq);
      fd.store(sd);
      if (tid < QB) {
        sl[buf][tid] = fl;
        se[buf][tid] = fe;
      }
      if constexpr (DIRECT) loads_done();
      __syncthreads();
      if (i + 1 < rep * tn) fetch(i + 1, 1 - buf);
      if (qb < ka || qa - kb >= a.window) continue;
      const bool full = qa >= kb && qb - ka < a.window;
#pragma unroll
      for (int qs = 0; qs < QB / 32; ++qs) {
        // sixteen queries at a time: their scores become halves of operands before the next ones' are formed
        Half<T> ph[2][KT], sh[2][KT];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int row = (qs * 2 + t) * 16;
          f32x4 s[KT], dp[KT];
#pragma unroll
          for (int kt = 0; kt < KT; ++kt) s[kt] = dp[kt] = zero4();
#pragma unroll
          for (int ds = 0; ds < DS; ++ds) {
            const Frag<T> qf = L::row(tq, row, ds * 32), df = L::row(td, row, ds * 32);
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
              s[kt] = mma(qf, kf[kt][ds], s[kt]);
              dp[kt] = mma(df, vf[kt][ds], dp[kt]);
            }
          }
          const f32x4 lse = *reinterpret_cast<const f32x4*>(&sl[buf][row + 4 * g4]), del = *reinterpret_cast<const f32x4*>(&se[buf][row + 4 * g4]);
#pragma unroll
          for (int kt = 0; kt < KT; ++kt) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int qi = qa + row + 4 * g4 + e, j = ka + kt * 16 + l16;
              float p = exp2_hw(fmaf(s[kt][e], scale2, -lse[e]));
              if (!full && !(j <= qi && qi - j < a.window)) p = 0.f;
              s[kt][e] = p;
              dp[kt][e] = p == 0.f ? 0.f : p * (dp[kt][e] - del[e]);
            }
            ph[t][kt] = to_half<T>(s[kt]);
            sh[t][kt] = to_half<T>(dp[kt]);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
        Frag<T> pf[KT], sf[KT];
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
          pf[kt] = __builtin_shufflevector(ph[0][kt], ph[1][kt], 0, 1, 2, 3, 4, 5, 6, 7);
          sf[kt] = __builtin_shufflevector(sh[0][kt], sh[1][kt], 0, 1, 2, 3, 4, 5, 6, 7);
        }
        auto product = [&](auto finite) __attribute__((always_inline)) {
#pragma unroll
          for (int d = 0; d < DT; ++d) {
            Frag<T> df = L::col(td, qs * 32, d * 16), qf = L::col(tq, qs * 32, d * 16);
            if constexpr (finite.value) {
              df = finite_only(df);
              qf = finite_only(qf);
              __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
              dv[d][kt] = mma(df, pf[kt], dv[d][kt]);
              dk[d][kt] = mma(qf, sf[kt], dk[d][kt]);
            }
          }
        };
        if (again.value && !full) product(again);
        else product(std::false_type());
      }
      if (again.value && !full) {
        auto seen = [&](int kt, int r) {
          const int qi = qa + r, j = ka + kt * 16 + l16;
          return qi < sp.len && j <= qi && qi - j < a.window;
        };
        add_not_finite<T, DP>(td, QB, dv, seen);
        add_not_finite<T, DP>(tq, QB, dk, seen);
      }
    }
    float sum = 0.f;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) sum = times_zero(dv[d][kt], times_zero(dk[d][kt], sum));
    return !again.value && any_not_finite(sum);
  };
  if (pass(std::false_type())) pass(std::true_type());
#pragma unroll
  for (int kt = 0; kt < KT; ++kt) {
    const int j = ka + kt * 16 + l16;
    if (j >= sp.len) continue;
    // the first keys' sums are added to those of the parts behind the window
    const bool later = j < a.sinks && sp.len > a.window;
    float* pw = later ? a.part + (((a.parts + sp.n) * a.sinks + j) * a.HK + hk) * 2 * a.D : nullptr;
    const int64_t row = ((sp.seq0 + j) * a.HK + hk) * a.D;
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      const int c = d * 16 + 4 * g4;
      if (c >= a.D) continue;
      const float x[4] = {dk[d][kt][0] * a.scale, dk[d][kt][1] * a.scale, dk[d][kt][2] * a.scale, dk[d][kt][3] * a.scale};
      const float y[4] = {dv[d][kt][0], dv[d][kt][1], dv[d][kt][2], dv[d][kt][3]};
      if (later) {
        store_n<float, 4>(pw + c, x, a.D - c, false);
        store_n<float, 4>(pw + a.D + c, y, a.D - c, false);
      } else {
        store_n<T, 4>(static_cast<T*>(a.dk) + row + c, x, a.D - c, VEC);
        store_n<T, 4>(static_cast<T*>(a.dv) + row + c, y, a.D - c, VEC);
      }
    }
  }
}

// Sixteen keys: of the first ones over a part of the queries behind the window, or, where there are few keys, any over the
// queries that see them through the window (NEAR). Each wave takes blocks of 32 queries of its own, through shared memory of
// its own, and the waves' sums are joined at the end. Queries of a part that see none of the sixteen first tokens but through the
// window are left out, or what is not finite in one that comes before a key would reach it (zero times an infinity). The others
// come behind all sixteen, unless the window has less than 15 tokens and first tokens go on behind it: SHORT, which looks
// at the blocks with such queries and forms them as the other kernels do.
template <class T, int DP>
constexpr int kKeysWaves = sizeof(T) * DP <= 512 ? 4 : 2;  // blocks of fp32 queries of 256 channels leave room for two
template <class T, int DP, int NW, bool VEC, bool SHORT, bool NEAR>
__global__ __launch_bounds__(64 * NW, sizeof(T) == 2 && DP <= 128 ? 2 : 1) void win_keys_kernel(WinArgs a) {
  constexpr int DS = DP / 32, DT = DP / 16, EV = 16 / (int)sizeof(T), PER = DP / EV, N = 32 * PER / 64;
  typedef Tile<T, DP> L;
  __shared__ __align__(16) T sq[NW][32 * L::LD], sd[NW][32 * L::LD];
  const int tid = threadIdx.x, lane = tid % 64, l16 = lane % 16, g4 = lane / 16;
  const int wave = __builtin_amdgcn_readfirstlane(tid / 64);
  const int rep = a.H / a.HK, ktiles = NEAR ? 1 : (a.sinks + 15) / 16;
  const int64_t per = NEAR ? a.blocks : a.parts, part = blockIdx.x % per;
  const int hk = (int)(blockIdx.x / per / ktiles);
  const Span sp = find_span(a.sq, NEAR ? 16 : a.part_len, (int)part, NEAR ? 0 : a.window);
  const int k0 = (NEAR ? sp.s : (int)(blockIdx.x / per % ktiles)) * 16;
  const int begin = NEAR ? k0 : a.window + sp.s * a.part_len, qlo = NEAR ? k0 : max(begin, k0 + a.window);
  const int qhi = NEAR ? (int)min((int64_t)sp.len, (int64_t)k0 + 15 + a.window) - 1 : min(begin + a.part_len, sp.len) - 1;
  if (begin >= sp.len) return;  // a sequence without tokens, or no longer than the window
  Frag<T> kf[DS], vf[DS];
  {
    const int j = k0 + l16;
    const bool in = j < sp.len && (NEAR || j < a.sinks);
    const T* k = static_cast<const T*>(a.k) + (sp.seq0 + j) * a.k_row + (int64_t)hk * a.D;
    const T* v = static_cast<const T*>(a.v) + (sp.seq0 + j) * a.v_row + (int64_t)hk * a.D;
#pragma unroll
    for (int s = 0; s < DS; ++s) {
      kf[s] = row_global<VEC>(k, s * 32, in ? a.D : 0);
      vf[s] = row_global<VEC>(v, s * 32, in ? a.D : 0);
    }
  }
  f32x4 dk[DT][1], dv[DT][1];
  const float scale2 = a.scale * kLog2e;
  const int nb = qhi < qlo ? 0 : (qhi - qlo) / 32 + 1;  // blocks of a head: none where the part ends before the tile's queries
  T *tq = sq[wave], *td = sd[wave];
  auto pass = [&](auto again) __attribute__((always_inline)) {
#pragma unroll
    for (int d = 0; d < DT; ++d) dk[d][0] = dv[d][0] = zero4();
    for (int b = wave; b < rep * nb; b += NW) {
      const int h = hk * rep + b / nb, q0 = qlo + b % nb * 32, rows = qhi - q0 + 1;
      const T* q = static_cast<const T*>(a.q) + (sp.seq0 + q0) * a.q_row + (int64_t)h * a.D;
      const T* d = static_cast<const T*>(a.dout) + ((sp.seq0 + q0) * a.H + h) * a.D;
      float lse2[2][4], delta[2][4];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = t * 16 + 4 * g4 + e;
          const int64_t row = (sp.seq0 + q0 + r) * a.H + h;
          lse2[t][e] = r < rows ? a.lse_in[row] * kLog2e : INFINITY;
          delta[t][e] = r < rows ? a.delta[row] : 0.f;
        }
      wave_sync();  // the last block has been read
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const T* from = half == 0 ? q : d;
        const int64_t row = half == 0 ? a.q_row : (int64_t)a.H * a.D;
        constexpr int BATCH = N < 4 ? N : 4;
#pragma unroll
        for (int i0 = 0; i0 < N; i0 += BATCH) {
          uint4 f[BATCH];
#pragma unroll
          for (int i = 0; i < BATCH; ++i) {
            const int id = lane + (i0 + i) * 64, r = id / PER, c = id % PER * EV;
            const auto x = load_n<T, EV>(from + r * row + c, r >= rows ? 0 : VEC ? (c < a.D ? EV : 0) : a.D - c, VEC);
            f[i] = make_uint4(x.w[0], x.w[1], x.w[2], x.w[3]);
            if constexpr (!VEC) asm volatile("" : "+v"(f[i].x), "+v"(f[i].y), "+v"(f[i].z), "+v"(f[i].w));
          }
#pragma unroll
          for (int i = 0; i < BATCH; ++i) {
            const int id = lane + (i0 + i) * 64;
            *reinterpret_cast<uint4*>((half == 0 ? tq : td) + L::block(id / PER, id % PER)) = f[i];
          }
          if constexpr (N > BATCH) wave_sync();  // one batch after the other: all at once would fill the registers
        }
      }
      wave_sync();
      const bool careful = NEAR ? again.value && !(q0 >= k0 + 15 && q0 + 31 - k0 < a.window)
                                : SHORT && q0 < k0 + 15 && (rows_not_finite<T, DP>(tq) || rows_not_finite<T, DP>(td));
      f32x4 s[2], dp[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        s[t] = dp[t] = zero4();
#pragma unroll
        for (int ds = 0; ds < DS; ++ds) {
          s[t] = mma(L::row(tq, t * 16, ds * 32), kf[ds], s[t]);
          dp[t] = mma(L::row(td, t * 16, ds * 32), vf[ds], dp[t]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int qi = q0 + t * 16 + 4 * g4 + e, j = k0 + l16;
          const bool seen = NEAR ? j <= qi && qi - j < a.window : qi - j >= a.window && j < a.sinks;
          const float p = seen ? exp2_hw(fmaf(s[t][e], scale2, -lse2[t][e])) : 0.f;
          s[t][e] = p;
          dp[t][e] = p == 0.f ? 0.f : p * (dp[t][e] - delta[t][e]);
        }
      }
      const Frag<T> pf = to_frag<T>(stack(s[0], s[1])), sf = to_frag<T>(stack(dp[0], dp[1]));
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) {
        Frag<T> df = L::col(td, 0, dt * 16), qf = L::col(tq, 0, dt * 16);
        if (careful) {
          df = finite_only(df);
          qf = finite_only(qf);
        }
        dv[dt][0] = mma(df, pf, dv[dt][0]);
        dk[dt][0] = mma(qf, sf, dk[dt][0]);
      }
      if (careful) {
        int c_tid = tid;
        if constexpr (SHORT) asm volatile("" : "+v"(c_tid));  // as in add_not_finite
        auto seen = [&](int, int r) {
          const int qi = q0 + r, j = k0 + c_tid % 16;
          return NEAR ? j <= qi && qi - j < a.window : qi - j >= a.window;
        };
        add_not_finite<T, DP>(td, 32, dv, seen);
        add_not_finite<T, DP>(tq, 32, dk, seen);
      }
    }
    if constexpr (NEAR && !again.value) {
      float sum = 0.f;
#pragma unroll
      for (int d = 0; d < DT; ++d) sum = times_zero(dv[d][0], times_zero(dk[d][0], sum));
      return any_not_finite(sum);
    } else {
      return false;
    }
  };
  // of the pairs that a part leaves out, the query sees the key through the window, or the block has been looked at
  if (pass(std::false_type())) pass(std::true_type());
  // the waves' sums, in order
  constexpr int LO = 2 * DP + 4;
  static_assert(sizeof(sq) >= 16 * LO * sizeof(float));
  float* so = reinterpret_cast<float*>(&sq[0][0]);
  __syncthreads();
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    if (wave == w) {
#pragma unroll
      for (int dt = 0; dt < DT; ++dt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float* p = so + l16 * LO + dt * 16 + 4 * g4 + e;
          p[0] = w == 0 ? dk[dt][0][e] * a.scale : fmaf(dk[dt][0][e], a.scale, p[0]);
          p[DP] = w == 0 ? dv[dt][0][e] : p[DP] + dv[dt][0][e];
        }
    }
    __syncthreads();
  }
  const int keys = min(16, (NEAR ? sp.len : min(a.sinks, sp.len)) - k0);
  for (int i = tid; i < keys * 2 * a.D; i += 64 * NW) {
    const int j = i / (2 * a.D), c = i % (2 * a.D);
    const float x = so[j * LO + (c < a.D ? c : DP + c - a.D)];
    if (!NEAR || (k0 + j < a.sinks && sp.len > a.window))  // parts, and the window's share behind them
      a.part[(((NEAR ? a.parts + sp.n : part) * a.sinks + k0 + j) * a.HK + hk) * 2 * a.D + c] = x;
    else
      static_cast<T*>(c < a.D ? a.dk : a.dv)[((sp.seq0 + k0 + j) * a.HK + hk) * a.D + c % a.D] = (T)x;
  }
}

template <class T, int DP, int QT, int MODE>
hipError_t win_fwd_t(const WinArgs& a, hipStream_t st) {
  hipLaunchKernelGGL((win_fwd_kernel<T, DP, QT, MODE>), dim3((uint32_t)(a.blocks * a.H)), dim3(256), 0, st, a);
  return hipGetLastError();
}
template <class T, int DP, int QT, int MODE>
hipError_t win_dq_t(const WinArgs& a, hipStream_t st) {
  hipLaunchKernelGGL((win_dq_kernel<T, DP, QT, MODE>), dim3((uint32_t)(a.blocks * a.H)), dim3(256), 0, st, a);
  return hipGetLastError();
}
template <class T, int DP, int KT, int MODE>
hipError_t win_dkv_t(const WinArgs& a, int krows, hipStream_t st) {
  constexpr int NW = kKeysWaves<T, DP>;
  if (krows == 16)
    hipLaunchKernelGGL((win_keys_kernel<T, DP, NW, MODE != kOdd, false, true>), dim3((uint32_t)(a.blocks * a.HK)), dim3(64 * NW), 0, st, a);
  else
    hipLaunchKernelGGL((win_dkv_kernel<T, DP, KT, MODE>), dim3((uint32_t)(a.blocks * a.HK)), dim3(256), 0, st, a);
  if (a.parts > 0) {
    const int64_t ktiles = (a.sinks + 15) / 16;
    const dim3 grid((uint32_t)(a.parts * ktiles * a.HK));
    if (a.window < 15 && a.sinks > a.window)
      hipLaunchKernelGGL((win_keys_kernel<T, DP, NW, MODE != kOdd, true, false>), grid, dim3(64 * NW), 0, st, a);
    else
      hipLaunchKernelGGL((win_keys_kernel<T, DP, NW, MODE != kOdd, false, false>), grid, dim3(64 * NW), 0, st, a);
  }
  return hipGetLastError();
}

}  // namespace kda
