// Linear attention: the scan over segments' states, the decays' gradients, sums over the heads of a group, the token step,
// and how sequences are cut.
#include <algorithm>

#include "mixer_device.h"

namespace kda {

// How the work is cut: tokens of a segment, and columns of a workgroup's tile (a wave for every 16; four where there are no more
// than 64, and in fp32, whose tiles fill the shared memory; else eight).
LinCut lin_cut(int dtype, int64_t longest, int64_t heads, int K, int V) {
  LinCut c;
  c.tile_k = dtype == KDA_BF16 && K > 64 ? 128 : 64;
  c.tile_v = dtype == KDA_BF16 && V > 64 ? 128 : 64;
  const int64_t groups = std::max<int64_t>(1, heads * ((V + c.tile_v - 1) / c.tile_v));
  auto cut = [&](int64_t want, int64_t least) {
    const int64_t n = (want + groups - 1) / groups;
    return (std::max((longest + n - 1) / n, least) + kLinChunk - 1) / kLinChunk * kLinChunk;
  };
  // Two workgroups for each CU, but segments of 256 tokens at least: below that their states are more bytes than their rows.
  // Where that leaves CUs without work, one workgroup each, of single chunks at least: a workgroup walks its chunks one after the
  // other, 2 to 3 us each (a training pass, us at least tokens 32, 64, 128, 256: 777 tokens of 4 heads in fp32 86, 97, 129, 202;
  // 300 of 4 heads 72, 77, 111, 162; 2 x 2048 of 8 heads 135, 135, 154, 192; 4096 of 8 heads of 256 channels, which is enough
  // work, 280 at 256 and 410 at 128).
  int64_t seg = cut(512, 256);
  if (groups * ((longest + seg - 1) / seg) < 256) seg = cut(256, kLinChunk);
  c.seg = (int)seg;
  return c;
}

namespace {

template <bool VEC>
hipError_t lin_walk(int dtype, int mode, const LinArgs& a, hipStream_t st) {
  if (dtype == KDA_F32) return lin_walk_f32<VEC>(mode, a, st);
  return mode == kLinDot || mode == kLinDotRev ? lin_walk_dot_bf16<VEC>(mode, a, st) : lin_walk_bf16<VEC>(mode, a, st);
}

}  // namespace

hipError_t launch_lin_walk(int dtype, int mode, const LinArgs& args, hipStream_t st) {
  LinArgs a = args;
  const uintptr_t all = reinterpret_cast<uintptr_t>(a.s0) | reinterpret_cast<uintptr_t>(a.fin) | reinterpret_cast<uintptr_t>(a.fin2) |
                        reinterpret_cast<uintptr_t>(a.copy0);
  a.svec = a.s_p == 1 && a.P % 4 == 0 && all % 16 == 0;
  return a.vec ? lin_walk<true>(dtype, mode, a, st) : lin_walk<false>(dtype, mode, a, st);
}

namespace {

// S_in of each segment from what the segments add: S <- decay S + added, elementwise over a state, in place. Backward, and
// where the forward's states are given, also the products <dS, S> at the segments' ends.
// E elements of a state a thread, the loads of AHEAD segments on their way together.
template <bool REV, int E, int AHEAD>
__global__ __launch_bounds__(256) void lin_scan_kernel(LinScanArgs a, int slices) {
  const int slice = blockIdx.x % slices, hv = blockIdx.x / slices % a.HV, n = blockIdx.x / slices / a.HV;
  // the sequence's first segment
  int first = 0, count;
  if (a.sq.cu == nullptr) {
    count = runs_of(a.sq.T, a.seg);
    first = n * count;
  } else {
    int part = 0;
    for (int i = threadIdx.x % 64; i < n; i += 64) part += runs_of(a.sq.cu[i + 1] - a.sq.cu[i], a.seg);
#pragma unroll
    for (int d = 1; d < 64; d *= 2) part += __shfl_xor(part, d);
    first = part;
    count = runs_of(a.sq.cu[n + 1] - a.sq.cu[n], a.seg);
  }
  __shared__ float red[4][AHEAD];
  const int64_t at = (int64_t)slice * 256 * E + threadIdx.x;
  float s[E];
  bool in[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    in[e] = at + e * 256 < a.KV;
    s[e] = in[e] && a.first != nullptr ? a.first[((int64_t)n * a.HV + hv) * a.KV + at + e * 256] : 0.f;
  }
  // segments in batches, whose loads are on their way together
  for (int k0 = 0; k0 < count; k0 += AHEAD) {
    float add[AHEAD][E], dec[AHEAD], dots[AHEAD];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      const int k = min(k0 + u, count - 1), seg = first + (REV ? count - 1 - k : k);
      dec[u] = 0.f;
      if (a.local) {
        dec[u] = a.seg_decay[(int64_t)seg * a.HV + hv];
        const float* p = a.states + ((int64_t)(REV ? seg : seg + n) * a.HV + hv) * a.KV + at;
#pragma unroll
        for (int e = 0; e < E; ++e) add[u][e] = in[e] ? p[e * 256] : 0.f;
      }
    }
    float f[REV ? AHEAD : 1][E];
    if (REV && a.fwd != nullptr) {
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        const int k = min(k0 + u, count - 1), seg = first + count - 1 - k;
        const float* p = a.fwd + ((int64_t)(seg + n + 1) * a.HV + hv) * a.KV + at;
#pragma unroll
        for (int e = 0; e < E; ++e) f[REV ? u : 0][e] = in[e] ? p[e * 256] : 0.f;
      }
    }
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      if (k0 + u >= count) break;
      const int seg = first + (REV ? count - 1 - k0 - u : k0 + u);
      if (REV && a.fwd != nullptr) {
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) sum = fmaf(s[e], f[REV ? u : 0][e], sum);
        dots[u] = group_sum<64>(sum);
      }
      if (a.local) {
        float* p = a.states + ((int64_t)(REV ? seg : seg + n) * a.HV + hv) * a.KV + at;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          if (in[e]) p[e * 256] = s[e];
          s[e] = fmaf(dec[u], s[e], add[u][e]);
        }
      }
    }
    if (REV && a.fwd != nullptr) {
      if (threadIdx.x % 64 == 0) {
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
          if (k0 + u < count) red[threadIdx.x / 64][u] = dots[u];
      }
      __syncthreads();
      const int u = threadIdx.x;
      if (u < AHEAD && k0 + u < count)
        a.dot[((int64_t)slice * a.nseg + first + count - 1 - k0 - u) * a.HV + hv] = (red[0][u] + red[1][u]) + (red[2][u] + red[3][u]);
      __syncthreads();
    }
  }
  if (!REV && a.local) {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (in[e]) a.states[((int64_t)(first + count + n) * a.HV + hv) * a.KV + at + e * 256] = s[e];
  }
  if (a.local && a.last != nullptr) {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (in[e]) a.last[((int64_t)n * a.HV + hv) * a.KV + at + e * 256] = s[e];
  }
}

// A decay's gradient is what all paths that cross its token give: for a segment, with X = <dS, S> at its end,
//   dg_t = X + sum_{i >= t} (q_i.dq_i - k_i.dk_i),
// in which a pair of tokens behind t counts once with each sign. Summed in 64 bits. The same from the segment's start is
// dg_t = X' - sum_{i < t} (...), with X' that of the segment before. The terms have fp32's errors, which add up over a segment, so
// what the two ends differ by is dealt out along it (1.0e-6 -> 7e-7 relative at segments of 1024 tokens).
__global__ __launch_bounds__(256) void lin_gate_kernel(LinGateArgs a) {
  __shared__ double sw[4];
  const int hv = blockIdx.x % a.HV, segidx = blockIdx.x / a.HV, tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
  const Span sp = find_span(a.sq, a.seg, segidx);
  const int begin = sp.s * a.seg, len = min(a.seg, sp.len - begin);
  const int64_t t0 = sp.seq0 + begin, total = a.sq.total;
  double x = 0.0;
  for (int64_t s = lane; s < a.slices; s += 64) x += (double)a.dots[(s * a.nseg + segidx) * a.HV + hv];
#pragma unroll
  for (int d = 1; d < 64; d *= 2) x += __shfl_xor(x, d);
  auto term = [&](int t) {
    double v = 0.0;
    if (t < len) {
      for (int i = 0; i < a.qtiles; ++i) v += (double)a.dotq[((int64_t)i * a.HV + hv) * total + t0 + t];
      for (int i = 0; i < a.ktiles; ++i) v -= (double)a.dotk[((int64_t)i * a.HV + hv) * total + t0 + t];
    }
    return v;
  };
  double apart = 0.0;  // what the ends differ by
  if (sp.s > 0) {
    double sum = 0.0;
    for (int t = tid; t < len; t += 256) sum += term(t);
    for (int64_t s = tid; s < a.slices; s += 256) sum -= (double)a.dots[(s * a.nseg + segidx - 1) * a.HV + hv];
#pragma unroll
    for (int d = 1; d < 64; d *= 2) sum += __shfl_xor(sum, d);
    if (lane == 0) sw[wave] = sum;
    __syncthreads();
    apart = x + ((sw[0] + sw[1]) + (sw[2] + sw[3]));
    __syncthreads();
  }
  double all = 0.0;
  for (int c = (len + 255) / 256 - 1; c >= 0; --c) {
    const int t = c * 256 + tid;
    double v = term(t);
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const double o = __shfl_down(v, d);
      if (lane + d < 64) v += o;
    }
    if (lane == 0) sw[wave] = v;
    __syncthreads();
    double later = x;
    for (int w = 3; w > wave; --w) later += sw[w];
    if (t < len) {
      const double dg = v + later - apart * ((double)(len - t) / len);
      if (a.part == nullptr) a.dg[(t0 + t) * a.HV + hv] = (float)dg;
      all += dg;
    }
    x += ((sw[3] + sw[2]) + sw[1]) + sw[0];
    __syncthreads();
  }
  if (a.part != nullptr) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) all += __shfl_xor(all, d);
    if (lane == 0) sw[wave] = all;
    __syncthreads();
    if (tid == 0) a.part[(int64_t)segidx * a.HV + hv] = (sw[0] + sw[1]) + (sw[2] + sw[3]);
  }
}

__global__ __launch_bounds__(64) void lin_gate_sum_kernel(const double* part, int64_t nseg, int HV, float* dg) {
  const int hv = blockIdx.x;
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < nseg; i += 64) s += part[i * HV + hv];
#pragma unroll
  for (int d = 1; d < 64; d *= 2) s += __shfl_xor(s, d);
  if (threadIdx.x == 0) dg[hv] = (float)s;
}

// Sums over the rep heads of a group. VEC elements of a head a thread.
template <class T, int VEC>
__global__ __launch_bounds__(256) void group_sum_kernel(const float* in, T* out, int64_t n, int rep, int W) {
  for (int64_t i = (blockIdx.x * (int64_t)256 + threadIdx.x) * VEC; i < n; i += (int64_t)gridDim.x * 256 * VEC) {
    const int64_t row = i / W;
    const float* p = in + row * rep * W + i % W;
    float s[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) s[e] = 0.f;
#pragma unroll 4
    for (int r = 0; r < rep; ++r) {
      const auto v = load_n<float, VEC>(p + (int64_t)r * W, VEC, true);
#pragma unroll
      for (int e = 0; e < VEC; ++e) s[e] += v.at(e);
    }
    store_n<T, VEC>(out + i, s, VEC, true);
  }
}

template <class T>
hipError_t group_sum_t(const float* in, void* out, int64_t rows, int rep, int W, hipStream_t st) {
  const bool vec = W % 4 == 0 && reinterpret_cast<uintptr_t>(out) % 16 == 0;
  const int64_t n = rows * W, per = vec ? 1024 : 256;
  const dim3 grid((uint32_t)std::min<int64_t>((n + per - 1) / per, 1 << 16));
  if (vec) hipLaunchKernelGGL((group_sum_kernel<T, 4>), grid, dim3(256), 0, st, in, static_cast<T*>(out), n, rep, W);
  else hipLaunchKernelGGL((group_sum_kernel<T, 1>), grid, dim3(256), 0, st, in, static_cast<T*>(out), n, rep, W);
  return hipGetLastError();
}

}  // namespace

int lin_scan_slice(int64_t segments) { return segments > 8 ? 256 : 1024; }
int64_t lin_scan_slices(int64_t KV, int slice) { return (KV + slice - 1) / slice; }

hipError_t launch_lin_scan(const LinScanArgs& a, bool rev, hipStream_t st) {
  const int slices = (int)lin_scan_slices(a.KV, a.slice);
  const dim3 grid((uint32_t)((int64_t)slices * a.HV * a.sq.n));
  if (a.slice == 256) {
    if (rev) hipLaunchKernelGGL((lin_scan_kernel<true, 1, 16>), grid, dim3(256), 0, st, a, slices);
    else hipLaunchKernelGGL((lin_scan_kernel<false, 1, 16>), grid, dim3(256), 0, st, a, slices);
  } else {
    if (rev) hipLaunchKernelGGL((lin_scan_kernel<true, 4, 4>), grid, dim3(256), 0, st, a, slices);
    else hipLaunchKernelGGL((lin_scan_kernel<false, 4, 4>), grid, dim3(256), 0, st, a, slices);
  }
  return hipGetLastError();
}

hipError_t launch_lin_gate(const LinGateArgs& a, hipStream_t st) {
  hipLaunchKernelGGL(lin_gate_kernel, dim3((uint32_t)(a.nseg * a.HV)), dim3(256), 0, st, a);
  if (a.part != nullptr) hipLaunchKernelGGL(lin_gate_sum_kernel, dim3(a.HV), dim3(64), 0, st, a.part, a.nseg, a.HV, a.dg);
  return hipGetLastError();
}

hipError_t launch_group_sum(int dtype, const float* in, void* out, int64_t rows, int rep, int W, hipStream_t st) {
  if (rows == 0) return hipSuccess;
  return dtype == KDA_F32 ? group_sum_t<float>(in, out, rows, rep, W, st) : group_sum_t<bf16>(in, out, rows, rep, W, st);
}

// ---- token step

namespace {

constexpr int CL = 8;             // lanes across the columns, four each
constexpr int GROUPS = 256 / CL;  // groups of lanes that the rows are dealt to

// As KDA's token step, without its second product: the state is read once and written once, S <- e^g S + k v^T, o = scale S^T q.
// KI rows a lane. VEC: rows and their tiles start on multiples of four elements.
template <class T, int KI, bool VEC>
__global__ __launch_bounds__(256) void lin_step_kernel(LinStepArgs a) {
  __shared__ float red[4][CL][4];
  const int tiles = (a.V + CL * 4 - 1) / (CL * 4);
  const int tile = blockIdx.x % tiles, hv = blockIdx.x / tiles, b = blockIdx.y;
  const int cl = threadIdx.x % CL, rg = threadIdx.x / CL;
  const int col = tile * CL * 4 + cl * 4, valid = a.V - col;
  // the state is on its way while the slot is checked
  const int asked = a.slots != nullptr ? a.slots[b] : b;
  const bool held = asked >= 0 && asked < a.slots_n;
  float* S = a.state + ((int64_t)(held ? asked : 0) * a.HV + hv) * a.K * a.V + col;
  float s[KI][4];
#pragma unroll
  for (int i = 0; i < KI; ++i) {
    const int r = rg + i * GROUPS;
    const bool in = held && r < a.K;
    if constexpr (VEC) {
      const float4 v = in && valid > 0 ? load_stream(S + (int64_t)r * a.V) : make_float4(0.f, 0.f, 0.f, 0.f);
      s[i][0] = v.x;
      s[i][1] = v.y;
      s[i][2] = v.z;
      s[i][3] = v.w;
    } else {
      const auto v = load_n<float, 4>(S + (int64_t)r * a.V, in ? valid : 0, false);
#pragma unroll
      for (int e = 0; e < 4; ++e) s[i][e] = v.at(e);
    }
  }
  const int slot = step_slot(a.slots, b, a.slots_n);
  T* o = static_cast<T*>(a.o) + ((int64_t)b * a.HV + hv) * a.V + col;
  if (slot < 0) {
    if (rg == 0 && valid > 0) {
      const float f = slot == -1 ? 0.f : __builtin_nanf("");
      const float out[4] = {f, f, f, f};
      store_n<T, 4>(o, out, valid, VEC);
    }
    return;
  }
  const int h = hv / (a.HV / a.H);
  const T* q = static_cast<const T*>(a.q) + b * a.q_row + (int64_t)h * a.K;
  const T* k = static_cast<const T*>(a.k) + b * a.k_row + (int64_t)h * a.K;
  const auto v4 = load_n<T, 4>(static_cast<const T*>(a.v) + b * a.v_row + (int64_t)hv * a.V + col, valid, VEC);
  const float g = a.g[a.g_const ? hv : (int64_t)b * a.HV + hv];
  const float decay = exp2_hw((g < -1e4f ? -1e4f : g) * kLog2e);
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < KI; ++i) {
    const int r = rg + i * GROUPS;
    const bool in = r < a.K;
    const float kk = in ? as_f(k[r]) : 0.f, qq = in ? as_f(q[r]) : 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      s[i][e] = fmaf(kk, v4.at(e), s[i][e] * decay);
      sum[e] = fmaf(qq, s[i][e], sum[e]);
    }
    if constexpr (VEC) {
      if (in && valid > 0) store_stream(S + (int64_t)r * a.V, make_float4(s[i][0], s[i][1], s[i][2], s[i][3]));
    } else {
      store_n<float, 4>(S + (int64_t)r * a.V, s[i], in ? valid : 0, false);
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    sum[e] += dpp<kRor8>(sum[e]);
    sum[e] = add_xor32(add_xor16(sum[e]));
  }
  if (threadIdx.x % 64 < CL) {
#pragma unroll
    for (int e = 0; e < 4; ++e) red[threadIdx.x / 64][cl][e] = sum[e];
  }
  __syncthreads();
  if (rg == 0 && valid > 0) {
    float out[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) out[e] = a.scale * ((red[0][cl][e] + red[1][cl][e]) + (red[2][cl][e] + red[3][cl][e]));
    store_n<T, 4>(o, out, valid, VEC);
  }
}

template <class T, int KI>
hipError_t lin_step_t(const LinStepArgs& a, hipStream_t st) {
  const dim3 grid((a.V + CL * 4 - 1) / (CL * 4) * a.HV, a.B);
  const bool vec = a.V % 4 == 0 && a.v_row % 4 == 0 && reinterpret_cast<uintptr_t>(a.state) % 16 == 0 &&
                   reinterpret_cast<uintptr_t>(a.v) % (4 * sizeof(T)) == 0 && reinterpret_cast<uintptr_t>(a.o) % (4 * sizeof(T)) == 0;
  if (vec) hipLaunchKernelGGL((lin_step_kernel<T, KI, true>), grid, dim3(256), 0, st, a);
  else hipLaunchKernelGGL((lin_step_kernel<T, KI, false>), grid, dim3(256), 0, st, a);
  return hipGetLastError();
}

template <class T>
hipError_t lin_step_k(const LinStepArgs& a, hipStream_t st) {
  if (a.K <= 32) return lin_step_t<T, 1>(a, st);
  if (a.K <= 64) return lin_step_t<T, 2>(a, st);
  if (a.K <= 128) return lin_step_t<T, 4>(a, st);
  return lin_step_t<T, 8>(a, st);
}

}  // namespace

hipError_t launch_lin_step(int dtype, const LinStepArgs& a, hipStream_t st) {
  return dtype == KDA_F32 ? lin_step_k<float>(a, st) : lin_step_k<bf16>(a, st);
}

}  // namespace kda
