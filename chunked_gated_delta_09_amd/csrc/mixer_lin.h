// Linear attention with a decay for each head: the walk over the chunks of a segment.
//
// With G_i the sum of a chunk's decays up to and including token i (in the exponent), whole = G_last, a chunk gives
//   o_i = scale e^{G_i} q_i S + sum_{j <= i} scale e^{G_i - G_j} (q_i.k_j) v_j,   S <- e^{whole} S + sum_j e^{whole - G_j} k_j v_j^T.
// The gradients are the same walk with other rows in the three places:
//   dq: forward in time, (x, y, z) = (do, v, k), state S^T;
//   dv: backward, (k, q, do), and dk: backward, (v, do, q), with the state's gradient dS and its transpose:
//   dk_j = e^{whole - G_j} v_j dS^T + sum_{i >= j} scale e^{G_i - G_j} (do_i.v_j) q_i,   dS <- e^{whole} dS + sum_i scale e^{G_i} q_i do_i^T.
// So one kernel does all four: out_i = in_i (x_i S) + sum_j pair_ij (x_i.y_j) z_j, S <- decay S + sum_j up_j y_j z_j^T.
// The decays are differences of G, never quotients of exponentials, so no gate is too strong; G is summed in 64 bits and
// held as two fp32 numbers, so that a strong gate among weak ones costs them nothing. A gate that is not finite (-infinity is the
// lowest of the finite ones) would make NaN of differences that do not cross it: it is left out of G, and a chunk's set of such
// tokens says which decays are NaN.
//
// A workgroup has one head's state for a tile of its columns: each of its waves holds [P, 16] in matrix results. Per chunk the
// waves share the pairs out among them (they go through shared memory, for all columns need them), then each forms its columns of
// the outputs and of the state. The state is its own operand (stacked order), x_i S and the pairs' products are formed
// transposed so that a lane has four neighbouring columns of a row to store, and up_j scales z's columns of the wave
// alone. The next chunk's rows are on their way meanwhile.
//
// Precision. q, k, v and do are exact operands. The state and its gradient are outputs in fp32, and the decays' gradients
// are differences of sums of products with them, so where those are formed what is rounded to bf16 is split into three
// terms first (exact): the scaled z columns and the state. Where outputs are bf16 themselves the state and the pairs take one term,
// 2^-9 relative for each product, as the output's own rounding, and the scaled z columns two, or their error would stay in the state
// (2.3e-3 relative against 64 bits where one term leaves 2.5e-3 and the output's rounding alone 1.7e-3, for 2 % of the time).
//
// Decays' gradients. With M_ij = pair_ij (q_i.k_j)(do_i.v_j), what a pair of a chunk gives, the walk of dq forms
// sum_j M_ij - sum_j M_ji for each token from both products in fp32 (so a pair's two signs cancel exactly), and adds
// q_i.dq_i of the state's part; the walk of dk gives k_i.dk_i of its state's part.
//
// Measured (B=4, T=4096, 32 value heads over 8 of 128 channels, bf16): states 66 and 69 us, o 116, dv 120, dq 181, dk 171. Of dq's the
// vector unit has work for 85 us (splitting, scaling, decays), the matrix unit for 45, shared memory for 52; they follow each other between
// the chunk's barriers, with four waves a SIMD to fill the gaps. 372 MB read and 271 written take 125 us at the rate of a copy.
#pragma once

#include "mixer_device.h"

namespace kda {

constexpr int kGateChunks = 8;  // chunks whose decays are summed at a time

__device__ __forceinline__ int64_t state_entry(int mode, const Span& sp, int segidx) {
  return mode == kStateSeq ? sp.n : mode == kStateSeg ? segidx : (int64_t)segidx + sp.n + (mode == kStateEnd);
}

// NU: terms of the scaled z columns.
template <class T, int PP, int NW, bool REV, bool OUT, bool DOT, int NU, bool VEC>
__global__ __launch_bounds__(64 * NW, PP <= 128 ? NW / 2 : NW / 4) void lin_walk_kernel(LinArgs a, int rtiles) {
  constexpr int CH = kLinChunk, PT = PP / 16, PS = PP / 32, IT = CH / 16, JS = CH / 32, NT = 64 * NW, RB = 16 * NW;
  constexpr bool B16 = sizeof(T) == 2;
  constexpr int NI = DOT && B16 ? 3 : 1;  // terms of the state
  constexpr int LX = PP + kPadCol<T>, LY = PP + kPadCol<T>, LZ = RB + kPadCol<T>, LP = CH + kPad<T>, LW = RB + kPadCol<T>;
  __shared__ __align__(16) T sx[OUT ? CH * LX : 8], sy[CH * LY], sz[CH * LZ], sw[DOT ? CH * LW : 8], sp_[OUT ? CH * LP : 8];
  __shared__ float sg[kGateChunks][4][CH];  // G in two parts, scale e^G, e^(whole - G)
  __shared__ float sdec[kGateChunks], sw_[OUT ? 1 : kGateChunks][2];  // e^whole; whole in two parts
  __shared__ uint32_t sbad[OUT ? kGateChunks : 1];  // a bit for each token whose gate is not finite
  __shared__ float red[DOT ? NW : 1][DOT ? CH : 1];
  __shared__ float sm[DOT && !REV ? IT * IT : 1][2][16];  // sums of M over a tile's earlier and later tokens

  const int tid = threadIdx.x, lane = tid % 64, l16 = lane % 16, g4 = lane / 16;
  const int wave = __builtin_amdgcn_readfirstlane(tid / 64);
  const int64_t id = xcd_order(blockIdx.x, gridDim.x);
  const int rt0 = (int)(id % rtiles), hv = (int)(id / rtiles % a.HV), segidx = (int)(id / rtiles / a.HV);
  const Span sp = find_span(a.sq, a.seg, segidx);
  const int begin = sp.s * a.seg, len = min(a.seg, sp.len - begin);
  const int64_t t0 = sp.seq0 + begin;
  const int hq = hv / a.rep, r0 = rt0 * RB;
  const int64_t KV = (int64_t)a.P * a.R;
  const int rcol = r0 + wave * 16 + l16;         // the lane's column of the state
  const int s_at = 4 * g4 * (int)a.s_p + rcol * (int)a.s_r;

  const T* x = static_cast<const T*>(a.x) + t0 * a.x_row + (int64_t)(a.x_qk ? hq : hv) * a.P;
  const T* y = static_cast<const T*>(a.y) + t0 * a.y_row + (int64_t)(a.y_qk ? hq : hv) * a.P;
  const T* z = static_cast<const T*>(a.z) + t0 * a.z_row + (int64_t)(a.z_qk ? hq : hv) * a.R + r0;
  const T* w = static_cast<const T*>(a.w) + t0 * a.w_row + (int64_t)(a.w_qk ? hq : hv) * a.R + r0;
  const int zw = a.R - r0;
  Stage<T, CH, PP, NT, VEC> fx, fy;
  Stage<T, CH, RB, NT, VEC> fz, fw;
  const int nc = (len + CH - 1) / CH;
  auto fetch = [&](int c) {
    const int rows = len - c * CH;
    const int64_t at = (int64_t)c * CH;
    if constexpr (OUT) fx.load(x + at * a.x_row, (int)a.x_row, rows, a.P);
    fy.load(y + at * a.y_row, (int)a.y_row, rows, a.P);
    fz.load(z + at * a.z_row, (int)a.z_row, rows, zw);
    if constexpr (DOT) fw.load(w + at * a.w_row, (int)a.w_row, rows, zw);
  };
  // The first rows and decays are on their way before the state's loads, which are waited for later.
  if (nc > 0) fetch(REV ? nc - 1 : 0);
  auto gate_of = [&](int t) { return t < len ? (a.g_const ? a.g[hv] : a.g[(t0 + t) * a.HV + hv]) : 0.f; };
  constexpr int GPER = 64 / CH;  // chunks whose decays a wave sums at a time
  static_assert(NW * GPER >= kGateChunks);
  float gt;
  auto gates = [&](int c) {
    int g_lane = lane;
    asm volatile("" : "+v"(g_lane));  // as in Stage
    const int k = wave * GPER + g_lane / CH;
    gt = k < kGateChunks ? gate_of((c / kGateChunks * kGateChunks + k) * CH + g_lane % CH) : 0.f;
  };
  if (nc > 0) gates(REV ? nc - 1 : 0);
  f32x4 S[PT];
  {
    const float* s0 = a.s0_mode == kStateNone ? nullptr : a.s0 + (state_entry(a.s0_mode, sp, segidx) * a.HV + hv) * KV;
    float* c0 = a.copy0 == nullptr ? nullptr : a.copy0 + (((int64_t)segidx + sp.n) * a.HV + hv) * KV;
    if (a.svec) {  // a lane's four rows lie side by side
#pragma unroll
      for (int pt = 0; pt < PT; ++pt) {
        const bool in = pt * 16 + 4 * g4 < a.P && rcol < a.R;
        S[pt] = in && s0 != nullptr ? *reinterpret_cast<const f32x4*>(s0 + pt * 16 + s_at) : zero4();
        if (in && c0 != nullptr) *reinterpret_cast<f32x4*>(c0 + pt * 16 + s_at) = S[pt];
      }
    } else {
#pragma unroll
      for (int pt = 0; pt < PT; ++pt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const bool in = pt * 16 + 4 * g4 + e < a.P && rcol < a.R;
          const int at = (pt * 16 + e) * (int)a.s_p + s_at;
          const float v = in && s0 != nullptr ? s0[at] : 0.f;
          S[pt][e] = v;
          if (in && c0 != nullptr) c0[at] = v;
        }
    }
  }
  if constexpr (OUT) {
    // pairs that the order of time leaves out stay zero where a product of 32 covers them
    for (int i = tid; i < CH * LP; i += NT) sp_[i] = (T)0.f;
  }
  double seg_sum = 0.0;

  for (int ci = 0; ci < nc; ++ci) {
    const int c = REV ? nc - 1 - ci : ci;
    __syncthreads();  // the last chunk's tiles have been read
    if (ci == 0 || c / kGateChunks != (REV ? c + 1 : c - 1) / kGateChunks) {
      if (ci > 0) gates(c);
      int g_lane = lane;
      asm volatile("" : "+v"(g_lane));  // as in Stage
      const int k = wave * GPER + g_lane / CH;
      static_assert(CH == 32);
      const bool odd = !(gt < INFINITY);
      const int i = g_lane % CH;
      const uint32_t bad = (uint32_t)(__ballot(odd) >> (g_lane - i));
      double v = (odd ? 0.0 : gt < -1e4f ? -1e4 : (double)gt) * 1.4426950408889634;
#pragma unroll
      for (int d = 1; d < CH; d *= 2) {
        const double o = __shfl_up(v, d, CH);
        if (i >= d) v += o;
      }
      const float hi = (float)v, rest = (float)(__shfl(v, CH - 1, CH) - v);
      if (k < kGateChunks) {
        sg[k][0][i] = hi;
        sg[k][1][i] = (float)(v - (double)hi);
        sg[k][2][i] = bad << (CH - 1 - i) ? __builtin_nanf("") : a.scale * exp2_hw(hi);
        sg[k][3][i] = bad >> i >> 1 ? __builtin_nanf("") : exp2_hw(rest);
        if (i == CH - 1) {
          if constexpr (OUT) {
            sbad[k] = bad;
          } else {
            sw_[k][0] = bad ? __builtin_nanf("") : hi;
            sw_[k][1] = (float)(v - (double)hi);
          }
          sdec[k] = bad ? __builtin_nanf("") : exp2_hw(hi);
        }
      }
    }
    if constexpr (OUT) fx.store_stacked(sx, LX);
    fy.store(sy, LY);
    fz.store(sz, LZ);
    if constexpr (DOT) fw.store(sw, LW);
    __syncthreads();
    if (ci + 1 < nc) fetch(REV ? c - 1 : c + 1);

    const int rows = len - c * CH;
    const float *gh = sg[c % kGateChunks][0], *gl = sg[c % kGateChunks][1];
    const float* in_w = sg[c % kGateChunks][REV ? 3 : 2];
    const float* up_w = sg[c % kGateChunks][REV ? 2 : 3];
    if constexpr (!OUT) seg_sum += (double)sw_[c % kGateChunks][0] + (double)sw_[c % kGateChunks][1];

    f32x4 o[IT];
    if constexpr (OUT) {
      // tiles of pairs, 16 later by 16 earlier tokens: a wave each
      if (wave < 3) {
        const int hi = wave < 2 ? 1 : 0, lo = wave == 1 ? 1 : 0, ti = REV ? lo : hi, tj = REV ? hi : lo;
        const int i = ti * 16 + l16;
        f32x4 acc = zero4(), bcc = zero4();
        const uint32_t bad = sbad[c % kGateChunks];
#pragma unroll
        for (int s = 0; s < PS; ++s) acc = mma(row_stk(sy + (tj * 16 + l16) * LY, s * 32), row_nat(sx + i * LX, s * 32), acc);
        if constexpr (DOT && !REV) {
          // z_j.w_i over the workgroup's columns
#pragma unroll
          for (int s = 0; s < RB / 32; ++s)
            bcc = mma(row_nat(sz + (tj * 16 + l16) * LZ, s * 32), row_nat(sw + i * LW, s * 32), bcc);
        }
        float p[4], m[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = tj * 16 + 4 * g4 + e;
          const float d = REV ? (gh[j] - gh[i]) + (gl[j] - gl[i]) : (gh[i] - gh[j]) + (gl[i] - gl[j]);
          p[e] = (REV ? j >= i : j <= i) ? acc[e] * (a.scale * exp2_hw(d)) : 0.f;
          m[e] = j < i ? p[e] * bcc[e] : 0.f;
        }
        store_n<T, 4>(sp_ + i * LP + stacked(tj * 16 + 4 * g4), p, 4, true);
        if (__builtin_expect(__builtin_amdgcn_readfirstlane((int)bad) != 0, 0)) {
          int b_lane = lane;
          asm volatile("" : "+v"(b_lane) : : "memory");  // as in Stage, and behind the store
#pragma unroll 1
          for (int e = 0; e < 4; ++e) {
            const int bi = ti * 16 + b_lane % 16, bj = tj * 16 + b_lane / 16 * 4 + e, from = min(bi, bj), to = max(bi, bj);
            if ((REV ? bj >= bi : bj <= bi) && (bad & ((2u << to) - (2u << from))) != 0)
              sp_[bi * LP + stacked(bj)] = (T)__builtin_nanf("");
          }
        }
        if constexpr (DOT && !REV) {
          const float over = add_xor32(add_xor16((m[0] + m[1]) + (m[2] + m[3])));
          float (*t)[16] = sm[ti * IT + tj];
          if (g4 == 0) t[0][l16] = over;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            m[e] = group_sum<16>(m[e]);
            if (l16 == 0) t[1][4 * g4 + e] = m[e];
          }
        }
      }
#pragma unroll
      for (int it = 0; it < IT; ++it) o[it] = zero4();
#pragma unroll
      for (int s = 0; s < PS; ++s) {
        Frag<T> sf[NI];
        split<T, NI>(stack(S[2 * s], S[2 * s + 1]), sf);
#pragma unroll
        for (int it = 0; it < IT; ++it) {
          const Frag<T> xf = row_nat(sx + (it * 16 + l16) * LX, s * 32);
#pragma unroll
          for (int n = NI - 1; n >= 0; --n) o[it] = mma(sf[n], xf, o[it]);
        }
      }
#pragma unroll
      for (int it = 0; it < IT; ++it) o[it] *= in_w[it * 16 + l16];
      if constexpr (DOT) {
        // the state's part of out_i.w_i
#pragma unroll
        for (int it = 0; it < IT; ++it) {
          const int i = it * 16 + l16;
          const auto wv = load_n<T, 4>(sw + i * LW + wave * 16 + 4 * g4, 4, true);  // zero behind the rows' ends
          float sum = 0.f;
#pragma unroll
          for (int e = 0; e < 4; ++e) sum = fmaf(wv.at(e), o[it][e], sum);
          sum = add_xor32(add_xor16(sum));
          if (g4 == 0) red[wave][i] = sum;
        }
      }
      __syncthreads();  // the pairs are there
    }
    // the state and, with the same columns of z, what the pairs give
    const float dec = sdec[c % kGateChunks];
#pragma unroll
    for (int pt = 0; pt < PT; ++pt) S[pt] *= dec;
    bool careful = false;
#pragma unroll
    for (int js = 0; js < JS; ++js) {
      Frag<T> zf = col_stk(sz, LZ, js * 32, wave * 16);
      Frag<T> uz[NU];
      const f32x4* up = reinterpret_cast<const f32x4*>(up_w + js * 32 + 4 * g4);
      split<T, NU>(to_f32<T>(zf) * stack(up[0], up[4]), uz);
      if constexpr (OUT) {
        // rows of z that are not finite reach only the tokens that see them: they are left out here and added below
        const f32x8 z8 = to_f32<T>(zf);
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) sum = fmaf(z8[e], 0.f, sum);
        if (__any(!(sum == 0.f))) {
          careful = true;
          zf = finite_only(zf);
        }
#pragma unroll
        for (int it = 0; it < IT; ++it) {
          if (REV ? js * 32 + 31 < it * 16 : js * 32 > it * 16 + 15) continue;
          o[it] = mma(zf, row_nat(sp_ + (it * 16 + l16) * LP, js * 32), o[it]);
        }
      }
#pragma unroll
      for (int pt = 0; pt < PT; ++pt) {
        const Frag<T> yf = col_stk(sy, LY, js * 32, pt * 16);
#pragma unroll
        for (int n = NU - 1; n >= 0; --n) S[pt] = mma(yf, uz[n], S[pt]);
      }
    }
    if constexpr (OUT) {
      int o_tid = threadIdx.x;
      asm volatile("" : "+v"(o_tid));  // as in Stage
      const int oi = o_tid % 16, og = o_tid % 64 / 16 * 4, ocol = r0 + wave * 16 + og;
      if (careful) {
#pragma unroll
        for (int it = 0; it < IT; ++it)
#pragma unroll 1
          for (int j = 0; j < CH; ++j) {
            const auto zr = load_n<T, 4>(sz + j * LZ + wave * 16 + og, 4, true);
            const int i = it * 16 + oi;
            const float p = (float)sp_[i * LP + stacked(j)];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if ((REV ? j >= i : j <= i) && !(fabsf(zr.at(e)) < INFINITY)) o[it][e] = fmaf(p, zr.at(e), o[it][e]);
          }
      }
      const int64_t oc = ((t0 + (int64_t)c * CH) * a.HV + hv) * a.R;
#pragma unroll
      for (int it = 0; it < IT; ++it) {
        const float v[4] = {o[it][0], o[it][1], o[it][2], o[it][3]};
        const uint32_t at = (uint32_t)(it * 16 + oi) * (uint32_t)(a.HV * a.R) + (uint32_t)ocol;
        if (it * 16 + oi < rows && ocol < a.R) {
          if (a.out_f32) store_n<float, 4>(static_cast<float*>(a.out) + oc + at, v, VEC ? 4 : a.R - ocol, VEC);
          else store_n<T, 4>(static_cast<T*>(a.out) + oc + at, v, VEC ? 4 : a.R - ocol, VEC);
        }
      }
      if constexpr (DOT) {
        if (tid < CH && tid < rows) {
          float d = 0.f;
#pragma unroll
          for (int n = 0; n < NW; ++n) d += red[n][tid];
          if constexpr (!REV) {
            const int t = tid / 16;
            for (int k = 0; k <= t; ++k) d += sm[t * IT + k][0][tid % 16];
            for (int k = t; k < IT; ++k) d -= sm[k * IT + t][1][tid % 16];
          }
          a.dot[((int64_t)rt0 * a.HV + hv) * a.sq.total + t0 + (int64_t)c * CH + tid] = d;
        }
      }
    }
  }

  // the state at the end; its offsets and bounds are formed anew, or they would be held all the way
  int e_tid = threadIdx.x;
  asm volatile("" : "+v"(e_tid));
  const int e_g = e_tid % 64 / 16 * 4, e_col = r0 + wave * 16 + e_tid % 16;
  const int e_at = e_g * (int)a.s_p + e_col * (int)a.s_r, e_p = e_col < a.R ? a.P - e_g : 0;
  for (int f = 0; f < 2; ++f) {
    float* fin = f == 0 ? a.fin : a.fin2;
    const int mode = f == 0 ? a.fin_mode : a.fin2_mode;
    if (fin == nullptr) continue;
    fin += (state_entry(mode, sp, segidx) * a.HV + hv) * KV;
    if (a.svec) {
#pragma unroll
      for (int pt = 0; pt < PT; ++pt)
        if (pt * 16 < e_p) *reinterpret_cast<f32x4*>(fin + pt * 16 + e_at) = S[pt];
      continue;
    }
#pragma unroll
    for (int pt = 0; pt < PT; ++pt)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (pt * 16 + e < e_p) fin[(pt * 16 + e) * (int)a.s_p + e_at] = S[pt][e];
  }
  if (!OUT && a.seg_decay != nullptr && rt0 == 0 && tid == 0)
    a.seg_decay[(int64_t)segidx * a.HV + hv] = exp2f((float)seg_sum);
}

template <class T, int PP, int NW, bool REV, bool OUT, bool DOT, int NU, bool VEC>
hipError_t lin_walk_t(const LinArgs& a, hipStream_t st) {
  const int rtiles = (a.R + 16 * NW - 1) / (16 * NW);
  hipLaunchKernelGGL((lin_walk_kernel<T, PP, NW, REV, OUT, DOT, NU, VEC>), dim3((uint32_t)(a.nseg * a.HV * rtiles)), dim3(64 * NW), 0,
                     st, a, rtiles);
  return hipGetLastError();
}

}  // namespace kda
