// One token of KDA for each sequence of a batch.
//
// A workgroup holds 32 columns of one head's state in registers (rows dealt to 32 groups of 8 lanes,
// four columns a lane), so the state is read once and written once: k^T S', q^T S' and q.k are summed
// together, u = beta (v - k^T S') follows, and o = scale (q^T S' + (q.k) u). Bound by the state's bytes.
#include "layer_device.h"

namespace kda {

namespace {

constexpr int kCols = 32;           // state columns of a workgroup
constexpr int kRowGroups = 32;      // 256 threads / 8 lanes of 4 columns

template <class T, int KI>
__global__ __launch_bounds__(256) void kda_step_kernel(KdaStepArgs a, int vec) {
  __shared__ float red[4][8][9];
  const int tiles = (a.V + kCols - 1) / kCols;
  const int tile = blockIdx.x % tiles, hv = blockIdx.x / tiles, b = blockIdx.y;
  const int slot = step_slot(a.slots, b, a.slots_n);
  const int cl = threadIdx.x % 8, rg = threadIdx.x / 8;
  const int col = tile * kCols + cl * 4, valid = a.V - col;
  T* o = static_cast<T*>(a.o) + ((int64_t)b * a.HV + hv) * a.V + col;
  if (slot < 0) {
    if (rg == 0 && valid > 0) {
      const float f = slot == -1 ? 0.f : __builtin_nanf("");
      const float out[4] = {f, f, f, f};
      store_n<T, 4>(o, out, valid, vec != 0);
    }
    return;
  }
  const int h = hv / (a.HV / a.H);
  float* S = a.state + ((int64_t)slot * a.HV + hv) * a.K * a.V + col;
  const T* q = static_cast<const T*>(a.q) + ((int64_t)b * a.H + h) * a.K;
  const T* k = static_cast<const T*>(a.k) + ((int64_t)b * a.H + h) * a.K;
  const float* g = a.g + ((int64_t)b * a.HV + hv) * a.K;
  float s[KI][4], kk[KI];
  Pack<float, 4> raw[KI];
#pragma unroll
  for (int i = 0; i < KI; ++i) {
    const int r = rg + i * kRowGroups;
    raw[i] = load_n<float, 4>(S + (int64_t)r * a.V, r < a.K ? valid : 0, vec != 0);
  }
  const auto v4 = load_n<T, 4>(static_cast<const T*>(a.v) + ((int64_t)b * a.HV + hv) * a.V + col, valid, vec != 0);
  float beta = a.beta[(int64_t)b * a.HV + hv];
  if (a.beta_logits) beta = sigmoid(beta);
  float sum[9];  // k^T S', q^T S' of four columns, q.k
#pragma unroll
  for (int e = 0; e < 9; ++e) sum[e] = 0.f;
#pragma unroll
  for (int i = 0; i < KI; ++i) {
    const int r = rg + i * kRowGroups;
    const bool in = r < a.K;
    kk[i] = in ? as_f(k[r]) : 0.f;
    const float qq = in ? as_f(q[r]) : 0.f;
    const float decay = in ? exp2_hw(g[r] * kLog2e) : 0.f;
    sum[8] = fmaf(qq, kk[i], sum[8]);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      s[i][e] = decay * raw[i].at(e);
      sum[e] = fmaf(kk[i], s[i][e], sum[e]);
      sum[4 + e] = fmaf(qq, s[i][e], sum[4 + e]);
    }
  }
#pragma unroll
  for (int e = 0; e < 9; ++e) {
    sum[e] += dpp<kRor8>(sum[e]);
    sum[e] = add_xor32(add_xor16(sum[e]));
  }
  if (threadIdx.x % 64 < 8) {
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
  if (rg == 0 && valid > 0) store_n<T, 4>(o, out, valid, vec != 0);
#pragma unroll
  for (int i = 0; i < KI; ++i) {
    const int r = rg + i * kRowGroups;
    float n[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) n[e] = fmaf(kk[i], u[e], s[i][e]);
    store_n<float, 4>(S + (int64_t)r * a.V, n, r < a.K ? valid : 0, vec != 0);
  }
}

template <class T, int KI>
hipError_t step_t(const KdaStepArgs& a, hipStream_t st) {
  const int tiles = (a.V + kCols - 1) / kCols;
  const bool vec = a.V % 4 == 0 && reinterpret_cast<uintptr_t>(a.state) % 16 == 0 &&
                   reinterpret_cast<uintptr_t>(a.v) % (4 * sizeof(T)) == 0 && reinterpret_cast<uintptr_t>(a.o) % (4 * sizeof(T)) == 0;
  hipLaunchKernelGGL((kda_step_kernel<T, KI>), dim3(tiles * a.HV, a.B), dim3(256), 0, st, a, (int)vec);
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
