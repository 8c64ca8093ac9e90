// Norm per group of channels with an activation, forward and backward.
//
// A group's C channels are held in registers by tpi lanes (a power of two up to a wave, or a whole
// workgroup), nch chunks of VEC elements each, so a row is read once: the mean, the centred sum of
// squares and the output come from the registers. Bound by memory.
#include "layer_device.h"

namespace kda {

namespace {

// Sum over the tpi lanes of a group. tpi = 256: the whole workgroup, through `sh` (4 floats; two
// buffers alternate, so one barrier a sum is enough).
__device__ __forceinline__ float item_sum(float x, int tpi, float* sh) {
  if (tpi >= 2) x += dpp<kXor1>(x);
  if (tpi >= 4) x += dpp<kXor2>(x);
  if (tpi >= 8) x += dpp<kHalfMirror>(x);
  if (tpi >= 16) x += dpp<kRor8>(x);
  if (tpi >= 32) x = add_xor16(x);
  if (tpi >= 64) x = add_xor32(x);
  if (tpi == 256) {
    if (threadIdx.x % 64 == 0) sh[threadIdx.x / 64] = x;
    __syncthreads();
    x = (sh[0] + sh[1]) + (sh[2] + sh[3]);
  }
  return x;
}

template <class T, int VEC, int NCH>
struct Row {
  float v[NCH][VEC];
};

template <class T, int VEC, int NCH>
__device__ __forceinline__ void load_row(const void* base, int64_t at, int C, int lane, int tpi, bool vec,
                                         float (&out)[NCH][VEC]) {
  const T* p = static_cast<const T*>(base) + at;
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int col = (c * tpi + lane) * VEC;
    const auto r = load_n<T, VEC>(p + col, C - col, vec);
#pragma unroll
    for (int e = 0; e < VEC; ++e) out[c][e] = as_f(r.v[e]);
  }
}

template <class T, int VEC, int NCH>
__device__ __forceinline__ void store_row(void* base, int64_t at, int C, int lane, int tpi, bool vec,
                                          const float (&in)[NCH][VEC]) {
  T* p = static_cast<T*>(base) + at;
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int col = (c * tpi + lane) * VEC;
    store_n<T, VEC>(p + col, in[c], C - col, vec);
  }
}

template <int VEC, int NCH>
__device__ __forceinline__ void load_param(const float* p, float fill, int64_t at, int C, int lane, int tpi,
                                           float (&out)[NCH][VEC]) {
#pragma unroll
  for (int c = 0; c < NCH; ++c)
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const int col = (c * tpi + lane) * VEC + e;
      out[c][e] = p != nullptr && col < C ? p[at + col] : fill;
    }
}

// x of a group -> n = (x - mean) rstd; returns rstd. Elements behind the group's end become zero.
template <int VEC, int NCH>
__device__ __forceinline__ float normalise(const NormArgs& a, int lane, int tpi, float* sh, float (&x)[NCH][VEC]) {
  const float inv = 1.f / (float)a.C;
  if (a.center) {
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int e = 0; e < VEC; ++e) s += x[c][e];
    const float mean = item_sum(s, tpi, sh) * inv;
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const int col = (c * tpi + lane) * VEC + e;
        x[c][e] = col < a.C ? x[c][e] - mean : 0.f;
      }
  }
  float q = 0.f;
#pragma unroll
  for (int c = 0; c < NCH; ++c)
#pragma unroll
    for (int e = 0; e < VEC; ++e) q = fmaf(x[c][e], x[c][e], q);
  const float rstd = 1.f / sqrtf(fmaf(item_sum(q, tpi, sh + 4), inv, a.eps));
#pragma unroll
  for (int c = 0; c < NCH; ++c)
#pragma unroll
    for (int e = 0; e < VEC; ++e) x[c][e] *= rstd;
  return rstd;
}

template <class T, int VEC, int NCH>
__global__ __launch_bounds__(256) void norm_fwd_kernel(NormArgs a, int tpi) {
  __shared__ float sh[8];
  const int lane = threadIdx.x % tpi;
  const int64_t item = (int64_t)blockIdx.x * (256 / tpi) + threadIdx.x / tpi;
  if (item >= a.R * a.G) return;  // whole groups of lanes leave; a workgroup-wide group always has its item
  const int64_t row = item / a.G;
  const int g = (int)(item % a.G);
  const bool vec = a.vec != 0;
  float x[NCH][VEC], gate[NCH][VEC], w[NCH][VEC], b[NCH][VEC];
  load_row<T, VEC, NCH>(a.x, row * a.x_row + (int64_t)g * a.C, a.C, lane, tpi, vec, x);
  if (a.gate != nullptr) load_row<T, VEC, NCH>(a.gate, row * a.gate_row + (int64_t)g * a.C, a.C, lane, tpi, vec, gate);
  const int64_t pat = a.shared ? 0 : (int64_t)g * a.C;
  load_param<VEC, NCH>(a.w, 1.f, pat, a.C, lane, tpi, w);
  load_param<VEC, NCH>(a.bias, 0.f, pat, a.C, lane, tpi, b);
  normalise<VEC, NCH>(a, lane, tpi, sh, x);
#pragma unroll
  for (int c = 0; c < NCH; ++c)
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float u = fmaf(x[c][e], w[c][e], b[c][e]);
      x[c][e] = a.gate != nullptr ? u * act_f(gate[c][e], a.act) : act_f(u, a.act);
    }
  store_row<T, VEC, NCH>(a.y, item * a.C, a.C, lane, tpi, vec, x);
}

// Backward. A group of lanes takes the items sub, sub + stride, ... with stride a multiple of G, so
// its channels (and the weights in its registers) stay the same and dweight, dbias are summed in
// registers. With du the gradient of u, dn = du w:
//   dx = rstd (dn - n mean(dn n) - [center] mean(dn)).
// Partial sums: one row a group of lanes [sub][2][C], or with one weight for all groups one row a
// workgroup.
template <class T, int VEC, int NCH>
__global__ __launch_bounds__(256) void norm_bwd_kernel(NormArgs a, int tpi, int64_t stride) {
  extern __shared__ float sh[];  // 16 floats, then [256 / tpi][C] where weights are shared
  const int lane = threadIdx.x % tpi, subs = 256 / tpi;
  const int64_t sub = (int64_t)blockIdx.x * subs + threadIdx.x / tpi;
  const int g = (int)(sub % a.G);
  const bool vec = a.vec != 0;
  const int64_t items = a.R * a.G;
  const float inv = 1.f / (float)a.C;
  float w[NCH][VEC], b[NCH][VEC], dw[NCH][VEC], db[NCH][VEC];
  const int64_t pat = a.shared ? 0 : (int64_t)g * a.C;
  load_param<VEC, NCH>(a.w, 1.f, pat, a.C, lane, tpi, w);
  load_param<VEC, NCH>(a.bias, 0.f, pat, a.C, lane, tpi, b);
#pragma unroll
  for (int c = 0; c < NCH; ++c)
#pragma unroll
    for (int e = 0; e < VEC; ++e) dw[c][e] = db[c][e] = 0.f;
  for (int64_t item = sub; item < items; item += stride) {
    const int64_t row = item / a.G;
    float x[NCH][VEC], gate[NCH][VEC], dy[NCH][VEC];
    load_row<T, VEC, NCH>(a.x, row * a.x_row + (int64_t)g * a.C, a.C, lane, tpi, vec, x);
    load_row<T, VEC, NCH>(a.dy, item * a.C, a.C, lane, tpi, vec, dy);
    if (a.gate != nullptr) load_row<T, VEC, NCH>(a.gate, row * a.gate_row + (int64_t)g * a.C, a.C, lane, tpi, vec, gate);
    const float rstd = normalise<VEC, NCH>(a, lane, tpi, sh, x);
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float u = fmaf(x[c][e], w[c][e], b[c][e]);
        float du;
        if (a.gate != nullptr) {
          const float z = gate[c][e];
          gate[c][e] = dy[c][e] * u * dact_f(z, a.act);
          du = dy[c][e] * act_f(z, a.act);
        } else {
          du = dy[c][e] * dact_f(u, a.act);
        }
        db[c][e] += du;
        dw[c][e] = fmaf(du, x[c][e], dw[c][e]);
        const float dn = du * w[c][e];
        dy[c][e] = dn;
        s1 += dn;
        s2 = fmaf(dn, x[c][e], s2);
      }
    if (a.gate != nullptr) store_row<T, VEC, NCH>(a.dgate, item * a.C, a.C, lane, tpi, vec, gate);
    s1 = a.center ? item_sum(s1, tpi, sh + 8) * inv : 0.f;
    s2 = item_sum(s2, tpi, sh + 12) * inv;
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int e = 0; e < VEC; ++e) x[c][e] = rstd * (dy[c][e] - s1 - x[c][e] * s2);
    store_row<T, VEC, NCH>(a.dx, item * a.C, a.C, lane, tpi, vec, x);
  }
  if (a.part == nullptr) return;
  if (!a.shared || subs == 1) {
    float* p = a.part + sub * 2 * a.C;
    if (!a.shared) p = a.part + ((sub / a.G) * 2 * a.G + g) * (int64_t)a.C;
    const int64_t second = a.shared ? a.C : (int64_t)a.G * a.C;
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const int col = (c * tpi + lane) * VEC + e;
        if (col < a.C) {
          p[col] = dw[c][e];
          p[second + col] = db[c][e];
        }
      }
    return;
  }
  float* acc = sh + 16;
  for (int k = 0; k < 2; ++k) {
    __syncthreads();
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const int col = (c * tpi + lane) * VEC + e;
        if (col < a.C) acc[(threadIdx.x / tpi) * a.C + col] = k == 0 ? dw[c][e] : db[c][e];
      }
    __syncthreads();
    for (int col = threadIdx.x; col < a.C; col += 256) {
      float s = 0.f;
      for (int r = 0; r < subs; ++r) s += acc[r * a.C + col];
      a.part[((int64_t)blockIdx.x * 2 + k) * a.C + col] = s;
    }
  }
}

// out[c] = sum_r in[r * stride + c]: 64 columns a workgroup, the rows dealt to 16 lanes a column
// (four running sums each) and joined in order.
__global__ __launch_bounds__(1024) void col_sum_kernel(const float* in, int64_t rows, int64_t cols, int64_t stride,
                                                       float* out) {
  __shared__ float sh[16][65];
  const int tx = threadIdx.x % 64, ty = threadIdx.x / 64;
  const int64_t col = (int64_t)blockIdx.x * 64 + tx;
  float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
  if (col < cols) {
    int64_t r = ty;
    for (; r + 48 < rows; r += 64) {
      s0 += in[r * stride + col];
      s1 += in[(r + 16) * stride + col];
      s2 += in[(r + 32) * stride + col];
      s3 += in[(r + 48) * stride + col];
    }
    for (; r < rows; r += 16) s0 += in[r * stride + col];
  }
  sh[ty][tx] = (s0 + s1) + (s2 + s3);
  __syncthreads();
  if (ty == 0 && col < cols) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) s += sh[i][tx];
    out[col] = s;
  }
}

template <class T, int VEC, int NCH>
hipError_t norm_fwd_t(const NormArgs& a, const NormPlan& p, hipStream_t st) {
  const int subs = 256 / p.tpi;
  const int64_t blocks = (a.R * a.G + subs - 1) / subs;
  hipLaunchKernelGGL((norm_fwd_kernel<T, VEC, NCH>), dim3((unsigned)blocks), dim3(256), 0, st, a, p.tpi);
  return hipGetLastError();
}

template <class T, int VEC, int NCH>
hipError_t norm_bwd_t(const NormArgs& a, const NormPlan& p, hipStream_t st) {
  const int subs = 256 / p.tpi;
  const size_t lds = sizeof(float) * (16 + (a.shared && subs > 1 ? (size_t)subs * a.C : 0));
  hipLaunchKernelGGL((norm_bwd_kernel<T, VEC, NCH>), dim3((unsigned)p.blocks), dim3(256), lds, st, a, p.tpi,
                     p.blocks * subs);
  return hipGetLastError();
}

#define NORM_DISPATCH(FN, T, VEC)                      \
  switch (p.nch) {                                     \
    case 1: return FN<T, VEC, 1>(a, p, st);            \
    case 2: return FN<T, VEC, 2>(a, p, st);            \
    case 4: return FN<T, VEC, 4>(a, p, st);            \
    default: return FN<T, VEC, 8>(a, p, st);           \
  }

}  // namespace

// Lanes of a group: enough for one chunk of 16 bytes each up to a wave, two chunks a lane up to
// 2 waves' worth, then the whole workgroup. Backward workgroups: about eight a CU, a whole number of
// rows' groups together (the lanes of a group stay on its channels), none without an item.
bool norm_plan(int dtype, int64_t R, int G, int C, int shared, NormPlan* p) {
  p->vec = dtype == KDA_F32 ? 4 : 8;
  const int chunks = (C + p->vec - 1) / p->vec;
  p->tpi = 1;
  while (p->tpi < 64 && p->tpi < chunks) p->tpi *= 2;
  if (chunks > 128) p->tpi = 256;
  p->nch = 1;
  while (p->nch * p->tpi < chunks) p->nch *= 2;
  if (p->nch > 8) return false;
  const int64_t subs = 256 / p->tpi;
  // workgroups in steps of G / gcd(G, subs)
  int64_t g = G, h = subs;
  while (h) {
    const int64_t r = g % h;
    g = h;
    h = r;
  }
  const int64_t step = G / g;
  const int64_t most = (R * G + subs - 1) / subs;
  int64_t blocks = (2048 + step - 1) / step * step;
  if (blocks > most) blocks = (most + step - 1) / step * step;
  p->blocks = blocks;
  p->part_cols = shared ? C : G * C;
  p->part_rows = shared ? blocks : blocks * subs / G;
  return true;
}

hipError_t launch_norm_fwd(int dtype, const NormArgs& a, hipStream_t st) {
  if (a.R == 0) return hipSuccess;
  NormPlan p;
  norm_plan(dtype, a.R, a.G, a.C, a.shared, &p);
  if (dtype == KDA_F32) {
    NORM_DISPATCH(norm_fwd_t, float, 4);
  }
  NORM_DISPATCH(norm_fwd_t, bf16, 8);
}

namespace {
hipError_t norm_bwd_main(int dtype, const NormArgs& a, const NormPlan& p, hipStream_t st) {
  if (dtype == KDA_F32) {
    NORM_DISPATCH(norm_bwd_t, float, 4);
  }
  NORM_DISPATCH(norm_bwd_t, bf16, 8);
}
}  // namespace

hipError_t launch_norm_bwd(int dtype, const NormArgs& a, hipStream_t st) {
  NormPlan p;
  norm_plan(dtype, a.R, a.G, a.C, a.shared, &p);
  if (a.R > 0) {
    const hipError_t e = norm_bwd_main(dtype, a, p, st);
    if (e != hipSuccess) return e;
  }
  const int64_t rows = a.R > 0 ? p.part_rows : 0;
  if (a.dw != nullptr) {
    const hipError_t e = launch_col_sum(a.part, rows, p.part_cols, 2 * (int64_t)p.part_cols, a.dw, st);
    if (e != hipSuccess) return e;
  }
  if (a.db != nullptr) return launch_col_sum(a.part + p.part_cols, rows, p.part_cols, 2 * (int64_t)p.part_cols, a.db, st);
  return hipSuccess;
}

hipError_t launch_col_sum(const float* in, int64_t rows, int64_t cols, int64_t stride, float* out, hipStream_t st) {
  hipLaunchKernelGGL(col_sum_kernel, dim3((unsigned)((cols + 63) / 64)), dim3(1024), 0, st, in, rows, cols, stride, out);
  return hipGetLastError();
}

}  // namespace kda
