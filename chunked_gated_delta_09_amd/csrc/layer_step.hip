// One token of KDA for each sequence of a batch.
//
// A workgroup holds a tile of columns of one head's state in registers (rows dealt to groups of lanes,
// four columns a lane), so the state is read once and written once: k^T S', q^T S' and q.k are summed
// together, u = beta (v - k^T S') follows, and o = scale (q^T S' + (q.k) u). Bound by the state's bytes:
// 256 sequences of 32 heads of 128 x 128 take 210 us for their 1.07 GB (5.1 TB/s; a large copy
// 5.2). Tiles of 32 columns: 64 or 128 columns a workgroup (longer pieces of a row, fewer workgroups) took 205 and
// 308 us where these took 207, and leave fewer workgroups to a small call.
#include "layer_device.h"

namespace kda {

namespace {

constexpr int CL = 8;            // lanes across the columns, four each
constexpr int GROUPS = 256 / CL;  // groups of lanes that the rows are dealt to

// KI rows a lane. VEC: rows and their tiles start on multiples of four elements.
template <class T, int KI, bool VEC>
__global__ __launch_bounds__(256) void kda_step_kernel(KdaStepArgs a) {
  __shared__ float red[4][CL][9];
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
  const T* q = static_cast<const T*>(a.q) + ((int64_t)b * a.H + h) * a.K;
  const T* k = static_cast<const T*>(a.k) + ((int64_t)b * a.H + h) * a.K;
  const float* g = a.g + ((int64_t)b * a.HV + hv) * a.K;
  float kk[KI];
  const auto v4 = load_n<T, 4>(static_cast<const T*>(a.v) + ((int64_t)b * a.HV + hv) * a.V + col, valid, VEC);
  float beta = a.beta[(int64_t)b * a.HV + hv];
  if (a.beta_logits) beta = sigmoid(beta);
  float sum[9];  // k^T S', q^T S' of four columns, q.k
#pragma unroll
  for (int e = 0; e < 9; ++e) sum[e] = 0.f;
#pragma unroll
  for (int i = 0; i < KI; ++i) {
    const int r = rg + i * GROUPS;
    const bool in = r < a.K;
    kk[i] = in ? as_f(k[r]) : 0.f;
    const float qq = in ? as_f(q[r]) : 0.f;
    const float decay = in ? exp2_hw(g[r] * kLog2e) : 0.f;
    sum[8] = fmaf(qq, kk[i], sum[8]);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      s[i][e] *= decay;
      sum[e] = fmaf(kk[i], s[i][e], sum[e]);
      sum[4 + e] = fmaf(qq, s[i][e], sum[4 + e]);
    }
  }
#pragma unroll
  for (int e = 0; e < 9; ++e) {
    sum[e] += dpp<kRor8>(sum[e]);
    sum[e] = add_xor32(add_xor16(sum[e]));
  }
  if (threadIdx.x % 64 < CL) {
#pragma unroll
    for (int e = 0; e < 9; ++e) red[threadIdx.x / 64][cl][e] = sum[e];
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < 9; ++e) sum[e] = (red[0][cl][e] + red[1][cl][e]) + (red[2][cl][e] + red[3][cl][e]);
  float u[4], out[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    u[e] = beta * (v4.at(e) - sum[e]);
    out[e] = a.scale * fmaf(sum[8], u[e], sum[4 + e]);
  }
  if (rg == 0 && valid > 0) store_n<T, 4>(o, out, valid, VEC);
#pragma unroll
  for (int i = 0; i < KI; ++i) {
    const int r = rg + i * GROUPS;
    float n[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) n[e] = fmaf(kk[i], u[e], s[i][e]);
    if constexpr (VEC) {
      if (r < a.K && valid > 0) store_stream(S + (int64_t)r * a.V, make_float4(n[0], n[1], n[2], n[3]));
    } else {
      store_n<float, 4>(S + (int64_t)r * a.V, n, r < a.K ? valid : 0, false);
    }
  }
}

template <class T, int KI>
hipError_t step_t(const KdaStepArgs& a, hipStream_t st) {
  const dim3 grid((a.V + CL * 4 - 1) / (CL * 4) * a.HV, a.B);
  const bool vec = a.V % 4 == 0 && reinterpret_cast<uintptr_t>(a.state) % 16 == 0 &&
                   reinterpret_cast<uintptr_t>(a.v) % (4 * sizeof(T)) == 0 && reinterpret_cast<uintptr_t>(a.o) % (4 * sizeof(T)) == 0;
  if (vec)
    hipLaunchKernelGGL((kda_step_kernel<T, KI, true>), grid, dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL((kda_step_kernel<T, KI, false>), grid, dim3(256), 0, st, a);
  return hipGetLastError();
}

template <class T>
hipError_t step_k(const KdaStepArgs& a, hipStream_t st) {
  if (a.K <= 32) return step_t<T, 1>(a, st);
  if (a.K <= 64) return step_t<T, 2>(a, st);
  if (a.K <= 128) return step_t<T, 4>(a, st);
  return step_t<T, 8>(a, st);
}

}  // namespace

hipError_t launch_kda_step(int dtype, const KdaStepArgs& a, hipStream_t st) {
  return dtype == KDA_F32 ? step_k<float>(a, st) : step_k<bf16>(a, st);
}

}  // namespace kda
