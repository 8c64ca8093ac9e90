// Norm per group of channels with an activation, forward and backward.
//
// A group's C channels are held in registers by tpi lanes (a power of two up to a wave, or a whole
// workgroup of 256 or 1024), one or two chunks of 16 bytes each, so a row is read once: the mean, the
// centred sum of squares and the output come from the registers. Bound by memory: 16384 rows of 32 x 128,
// bf16, gated, move their 403 MB forward in 81 us (5.0 TB/s; a large copy 5.2) and their 671 MB backward in
// 128 (5.2).
#include "layer_device.h"

namespace kda {

namespace {

// Sum over the tpi lanes of a group. tpi > 64: the whole workgroup, through `sh` (a float for each wave;
// the sums of an item have places of their own, so one barrier a sum is enough).
__device__ __forceinline__ float item_sum(float x, int tpi, float* sh) {
  if (tpi >= 2) x += dpp<kXor1>(x);
  if (tpi >= 4) x += dpp<kXor2>(x);
  if (tpi >= 8) x += dpp<kHalfMirror>(x);
  if (tpi >= 16) x += dpp<kRor8>(x);
  if (tpi >= 32) x = add_xor16(x);
  if (tpi >= 64) x = add_xor32(x);
  if (tpi > 64) {
    if (threadIdx.x % 64 == 0) sh[threadIdx.x / 64] = x;
    __syncthreads();
    x = 0.f;
    for (int i = 0; i < tpi / 64; ++i) x += sh[i];
  }
  return x;
}

// Where a lane's elements are in its group. NEAR (C a multiple of VEC): VEC neighbours a chunk, loaded
// together where rows are aligned for it (`vec`). Otherwise neighbouring lanes have neighbouring
// elements, so that loads and stores of single elements cover whole lines (1500 rows of 3 x 333, fp32:
// forward 6.7 against 10.4 us, backward 13.8 against 17.5). The choice goes by C alone: the order of a group's sums, and with it its bits, does
// not depend on where the tensor lies.
template <int VEC, bool NEAR>
struct Place {
  int lane, tpi, C;
  bool vec;
  __device__ __forceinline__ int col(int c, int e) const {
    return NEAR ? (c * tpi + lane) * VEC + e : (c * VEC + e) * tpi + lane;
  }
  __device__ __forceinline__ bool has(int c, int e) const { return NEAR ? col(c, 0) < C : col(c, e) < C; }
};

// A lane's share of a group, as loaded; zero behind the group's end.
template <class T, int VEC, int NCH>
struct Raw {
  Pack<T, VEC> v[NCH];

  template <bool NEAR>
  __device__ __forceinline__ void load(const void* base, int64_t at, const Place<VEC, NEAR>& pl) {
    const T* p = static_cast<const T*>(base) + at;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      if constexpr (NEAR) {
        v[c] = load_n<T, VEC>(p + pl.col(c, 0), pl.has(c, 0) ? VEC : 0, pl.vec);
      } else {
#pragma unroll
        for (int i = 0; i < Pack<T, VEC>::WORDS; ++i) v[c].w[i] = 0;
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          if (pl.has(c, e)) v[c].put(e, p[pl.col(c, e)]);
      }
    }
  }
  __device__ __forceinline__ float at(int c, int e) const { return v[c].at(e); }
};

// The activation of a call, without branches for its elements.
struct Act {
  bool none, silu;
  __device__ __forceinline__ explicit Act(int act) : none(act == KDA_ACT_NONE), silu(act == KDA_ACT_SILU) {}
  __device__ __forceinline__ float value(float x) const {
    const float v = sigmoid(x) * (silu ? x : 1.f);
    return none ? x : v;
  }
  // value and derivative
  __device__ __forceinline__ float both(float x, float* d) const {
    const float s = sigmoid(x), r = 1.f - s;
    const float v = s * (silu ? x : 1.f), g = s * (silu ? fmaf(x, r, 1.f) : r);
    *d = none ? 1.f : g;
    return none ? x : v;
  }
};

template <class T, int VEC, int NCH, bool NEAR>
__device__ __forceinline__ void store_row(void* base, int64_t at, const Place<VEC, NEAR>& pl, const float (&in)[NCH][VEC]) {
  T* p = static_cast<T*>(base) + at;
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    if constexpr (NEAR) {
      store_n<T, VEC>(p + pl.col(c, 0), in[c], pl.has(c, 0) ? VEC : 0, pl.vec);
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (pl.has(c, e)) p[pl.col(c, e)] = (T)in[c][e];
    }
  }
}

template <int VEC, int NCH, bool NEAR>
__device__ __forceinline__ void load_param(const float* p, float fill, int64_t at, const Place<VEC, NEAR>& pl, bool vec,
                                           float (&out)[NCH][VEC]) {
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    if (NEAR && p != nullptr && vec && pl.has(c, 0)) {
#pragma unroll
      for (int e = 0; e < VEC; e += 4) {
        const float4 v = *reinterpret_cast<const float4*>(p + at + pl.col(c, 0) + e);
        out[c][e] = v.x;
        out[c][e + 1] = v.y;
        out[c][e + 2] = v.z;
        out[c][e + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) out[c][e] = p != nullptr && pl.has(c, e) ? p[at + pl.col(c, e)] : fill;
    }
  }
}

// x of a group -> n = (x - mean) rstd; returns rstd. Elements behind the group's end become zero.
template <int VEC, int NCH, bool NEAR>
__device__ __forceinline__ float normalise(const NormArgs& a, const Place<VEC, NEAR>& pl, float* sh, float (&x)[NCH][VEC]) {
  const float inv = 1.f / (float)a.C;
  if (a.center) {
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int e = 0; e < VEC; ++e) s += x[c][e];
    const float mean = item_sum(s, pl.tpi, sh) * inv;
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        x[c][e] = pl.has(c, e) ? x[c][e] - mean : 0.f;
      }
  }
  float q = 0.f;
#pragma unroll
  for (int c = 0; c < NCH; ++c)
#pragma unroll
    for (int e = 0; e < VEC; ++e) q = fmaf(x[c][e], x[c][e], q);
  const float rstd = 1.f / sqrtf(fmaf(item_sum(q, pl.tpi, sh + 16), inv, a.eps));
#pragma unroll
  for (int c = 0; c < NCH; ++c)
#pragma unroll
    for (int e = 0; e < VEC; ++e) x[c][e] *= rstd;
  return rstd;
}

// A group of lanes takes the items sub, sub + stride, ... with stride a multiple of G, so its channels
// (and the weights in its registers) stay the same; the next item is loaded while this one is worked on. The
// last workgroup may have groups of lanes behind the stride: they take none.
template <class T, int VEC, int NCH, int THREADS, bool NEAR>
__global__ __launch_bounds__(THREADS) void norm_fwd_kernel(NormArgs a, int tpi, int64_t stride) {
  __shared__ float sh[32];
  const int lane = threadIdx.x % tpi;
  const int64_t sub = (int64_t)blockIdx.x * (THREADS / tpi) + threadIdx.x / tpi;
  if (sub >= stride) return;  // whole groups of lanes leave; a workgroup-wide group always has its item
  const int g = (int)(sub % a.G);
  const Place<VEC, NEAR> pl{lane, tpi, a.C, a.vec != 0};
  const int64_t pat = a.shared ? 0 : (int64_t)g * a.C, step = stride / a.G;
  int64_t row = sub / a.G;
  Raw<T, VEC, NCH> rx, rg;
  rx.load(a.x, row * a.x_row + (int64_t)g * a.C, pl);
  if (a.gate != nullptr) rg.load(a.gate, row * a.gate_row + (int64_t)g * a.C, pl);
  float w[NCH][VEC], b[NCH][VEC];
  load_param<VEC, NCH, NEAR>(a.w, 1.f, pat, pl, a.wvec != 0, w);
  load_param<VEC, NCH, NEAR>(a.bias, 0.f, pat, pl, a.wvec != 0, b);
  const Act act(a.act);
  for (; row < a.R; row += step) {
    float x[NCH][VEC];
    const Raw<T, VEC, NCH> kg = rg;
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int e = 0; e < VEC; ++e) x[c][e] = rx.at(c, e);
    if (row + step < a.R) {
      rx.load(a.x, (row + step) * a.x_row + (int64_t)g * a.C, pl);
      if (a.gate != nullptr) rg.load(a.gate, (row + step) * a.gate_row + (int64_t)g * a.C, pl);
    }
    normalise<VEC, NCH, NEAR>(a, pl, sh, x);
    if (a.gate != nullptr) {
#pragma unroll
      for (int c = 0; c < NCH; ++c)
#pragma unroll
        for (int e = 0; e < VEC; ++e) x[c][e] = fmaf(x[c][e], w[c][e], b[c][e]) * act.value(kg.at(c, e));
    } else {
#pragma unroll
      for (int c = 0; c < NCH; ++c)
#pragma unroll
        for (int e = 0; e < VEC; ++e) x[c][e] = act.value(fmaf(x[c][e], w[c][e], b[c][e]));
    }
    store_row<T, VEC, NCH, NEAR>(a.y, (row * a.G + g) * a.C, pl, x);
    if (tpi > 64) __syncthreads();  // the sums' places are read before the next item's are written
  }
}

// Backward, items dealt as above: dweight and dbias are summed in registers. With du the gradient of u, dn = du w:
//   dx = rstd (dn - n mean(dn n) - [center] mean(dn)).
// Partial sums: one row a group of lanes [sub][2][C], or with one weight for all groups one row a
// workgroup.
template <class T, int VEC, int NCH, int THREADS, bool NEAR>
__global__ __launch_bounds__(THREADS) void norm_bwd_kernel(NormArgs a, int tpi, int64_t stride) {
  extern __shared__ float sh[];  // 64 floats, then [groups of lanes][C] where weights are shared
  const int lane = threadIdx.x % tpi, subs = THREADS / tpi;
  const int64_t sub = (int64_t)blockIdx.x * subs + threadIdx.x / tpi;
  const int g = (int)(sub % a.G);
  const Place<VEC, NEAR> pl{lane, tpi, a.C, a.vec != 0};
  const int64_t step = stride / a.G;
  const float inv = 1.f / (float)a.C;
  float w[NCH][VEC], b[NCH][VEC], dw[NCH][VEC], db[NCH][VEC];
  const int64_t pat = a.shared ? 0 : (int64_t)g * a.C;
  const bool used = sub < stride;
  int64_t row = used ? sub / a.G : a.R;
  Raw<T, VEC, NCH> rx, rg, rd;
  auto fetch = [&](int64_t r) {
    rx.load(a.x, r * a.x_row + (int64_t)g * a.C, pl);
    rd.load(a.dy, (r * a.G + g) * a.C, pl);
    if (a.gate != nullptr) rg.load(a.gate, r * a.gate_row + (int64_t)g * a.C, pl);
  };
  if (used) fetch(row);
  load_param<VEC, NCH, NEAR>(a.w, 1.f, pat, pl, a.wvec != 0, w);
  load_param<VEC, NCH, NEAR>(a.bias, 0.f, pat, pl, a.wvec != 0, b);
  const Act act(a.act);
#pragma unroll
  for (int c = 0; c < NCH; ++c)
#pragma unroll
    for (int e = 0; e < VEC; ++e) dw[c][e] = db[c][e] = 0.f;
  for (; row < a.R; row += step) {
    float x[NCH][VEC], dn[NCH][VEC];
    const Raw<T, VEC, NCH> kd = rd, kg = rg;
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int e = 0; e < VEC; ++e) x[c][e] = rx.at(c, e);
    if (row + step < a.R) fetch(row + step);
    const float rstd = normalise<VEC, NCH, NEAR>(a, pl, sh, x);
    const int64_t out = (row * a.G + g) * a.C;
    float s1 = 0.f, s2 = 0.f;
    if (a.gate != nullptr) {
      float dg[NCH][VEC];
#pragma unroll
      for (int c = 0; c < NCH; ++c)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          float d;
          const float dy = kd.at(c, e), v = act.both(kg.at(c, e), &d);
          dg[c][e] = dy * fmaf(x[c][e], w[c][e], b[c][e]) * d;
          dn[c][e] = dy * v;
        }
      store_row<T, VEC, NCH, NEAR>(a.dgate, out, pl, dg);
    } else {
#pragma unroll
      for (int c = 0; c < NCH; ++c)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          float d;
          act.both(fmaf(x[c][e], w[c][e], b[c][e]), &d);
          dn[c][e] = kd.at(c, e) * d;
        }
    }
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        db[c][e] += dn[c][e];
        dw[c][e] = fmaf(dn[c][e], x[c][e], dw[c][e]);
        dn[c][e] *= w[c][e];
        s1 += dn[c][e];
        s2 = fmaf(dn[c][e], x[c][e], s2);
      }
    s1 = a.center ? item_sum(s1, tpi, sh + 32) * inv : 0.f;
    s2 = item_sum(s2, tpi, sh + 48) * inv;
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int e = 0; e < VEC; ++e) x[c][e] = rstd * (dn[c][e] - s1 - x[c][e] * s2);
    store_row<T, VEC, NCH, NEAR>(a.dx, out, pl, x);
  }
  if (a.part == nullptr) return;
  if (!a.shared || subs == 1) {
    if (!used) return;
    float* p = a.part + sub * 2 * a.C;
    if (!a.shared) p = a.part + ((sub / a.G) * 2 * a.G + g) * (int64_t)a.C;
    const int64_t second = a.shared ? a.C : (int64_t)a.G * a.C;
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const int col = pl.col(c, e);
        if (pl.has(c, e)) {
          p[col] = dw[c][e];
          p[second + col] = db[c][e];
        }
      }
    return;
  }
  float* acc = sh + 64;
  for (int k = 0; k < 2; ++k) {
    __syncthreads();
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        if (pl.has(c, e)) acc[(threadIdx.x / tpi) * a.C + pl.col(c, e)] = k == 0 ? dw[c][e] : db[c][e];
      }
    __syncthreads();
    for (int col = threadIdx.x; col < a.C; col += THREADS) {
      float s = 0.f;
      for (int r = 0; r < subs; ++r) s += acc[r * a.C + col];
      a.part[((int64_t)blockIdx.x * 2 + k) * a.C + col] = s;
    }
  }
}

// out0[c], out1[c] = sum_r in[r][0][c], in[r][1][c]: 16 columns a workgroup, the rows dealt to 64 lanes a
// column (four running sums each) and joined in a fixed order.
__global__ __launch_bounds__(1024) void col_sum_kernel(const float* in, int64_t rows, int64_t cols, float* out0,
                                                       float* out1) {
  __shared__ float sh[64][17];
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const int64_t col = (int64_t)blockIdx.x * 16 + tx, stride = 2 * cols;
  float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
  if (col < stride) {
    int64_t r = ty;
    for (; r + 192 < rows; r += 256) {
      s0 += in[r * stride + col];
      s1 += in[(r + 64) * stride + col];
      s2 += in[(r + 128) * stride + col];
      s3 += in[(r + 192) * stride + col];
    }
    for (; r < rows; r += 64) s0 += in[r * stride + col];
  }
  sh[ty][tx] = (s0 + s1) + (s2 + s3);
  for (int half = 32; half > 0; half /= 2) {
    __syncthreads();
    if (ty < half) sh[ty][tx] += sh[ty + half][tx];
  }
  if (ty == 0 && col < stride) {
    float* out = col < cols ? out0 : out1;
    if (out != nullptr) out[col < cols ? col : col - cols] = sh[0][tx];
  }
}

template <class T, int VEC, int NCH, int THREADS>
hipError_t norm_fwd_t(const NormArgs& a, const NormPlan& p, hipStream_t st) {
  const dim3 grid((unsigned)p.blocks), block(THREADS);
  if (a.C % VEC == 0)
    hipLaunchKernelGGL((norm_fwd_kernel<T, VEC, NCH, THREADS, true>), grid, block, 0, st, a, p.tpi, p.stride);
  else
    hipLaunchKernelGGL((norm_fwd_kernel<T, VEC, NCH, THREADS, false>), grid, block, 0, st, a, p.tpi, p.stride);
  return hipGetLastError();
}

template <class T, int VEC, int NCH, int THREADS>
hipError_t norm_bwd_t(const NormArgs& a, const NormPlan& p, hipStream_t st) {
  const int subs = THREADS / p.tpi;
  const size_t lds = sizeof(float) * (64 + (a.shared && subs > 1 ? (size_t)subs * a.C : 0));
  const dim3 grid((unsigned)p.blocks), block(THREADS);
  if (a.C % VEC == 0)
    hipLaunchKernelGGL((norm_bwd_kernel<T, VEC, NCH, THREADS, true>), grid, block, lds, st, a, p.tpi, p.stride);
  else
    hipLaunchKernelGGL((norm_bwd_kernel<T, VEC, NCH, THREADS, false>), grid, block, lds, st, a, p.tpi, p.stride);
  return hipGetLastError();
}

// A bf16 group of 1024 lanes never needs a second chunk: 8192 channels are one each.
#define NORM_DISPATCH(FN)                                                    \
  do {                                                                       \
    if (dtype == KDA_F32) {                                                  \
      if (p.tpi == 1024)                                                     \
        return p.nch == 1 ? FN<float, 4, 1, 1024>(a, p, st) : FN<float, 4, 2, 1024>(a, p, st); \
      return p.nch == 1 ? FN<float, 4, 1, 256>(a, p, st) : FN<float, 4, 2, 256>(a, p, st);     \
    }                                                                        \
    if (p.tpi == 1024) return FN<bf16, 8, 1, 1024>(a, p, st);                \
    return p.nch == 1 ? FN<bf16, 8, 1, 256>(a, p, st) : FN<bf16, 8, 2, 256>(a, p, st);         \
  } while (0)

}  // namespace

// Lanes of a group: enough for one chunk of 16 bytes each up to a wave, for two chunks up to two waves'
// worth, then a workgroup of 256 and of 1024 in the same way. Workgroups: up to eight a CU of 256, taking
// whole rows side by side (the lanes of a group stay on its channels); a row of more groups than that has
// workgroups for all of them.
bool norm_plan(int dtype, int64_t R, int G, int C, int shared, bool bwd, NormPlan* p) {
  p->vec = dtype == KDA_F32 ? 4 : 8;
  const int chunks = (C + p->vec - 1) / p->vec;
  p->tpi = 1;
  while (p->tpi < 64 && p->tpi < chunks) p->tpi *= 2;
  if (chunks > 128) p->tpi = 256;
  if (chunks > 512) p->tpi = 1024;
  p->nch = chunks > p->tpi ? 2 : 1;
  if (chunks > 2 * p->tpi) return false;
  const int64_t subs = p->tpi == 1024 ? 1 : 256 / p->tpi;
  const int64_t most = (R * G + subs - 1) / subs;
  int64_t full = p->tpi == 1024 ? 512 : 2048;
  if (bwd) {
    // each workgroup leaves a row of sums: at least four items a group of lanes, but for a small call
    full /= 2;
    if (most / 4 < full) full = most / 4 > 256 ? most / 4 : 256;
  }
  // rows whose groups are taken side by side: as many as fill those workgroups, rounded up, and there are
  int64_t rows = (full * subs + G - 1) / G;
  if (rows > R) rows = R;
  p->stride = rows * G;
  p->blocks = (p->stride + subs - 1) / subs;
  p->part_cols = shared ? C : G * C;
  p->part_rows = shared ? p->blocks : rows;
  return true;
}

hipError_t launch_norm_fwd(int dtype, const NormArgs& a, hipStream_t st) {
  if (a.R == 0) return hipSuccess;
  NormPlan p;
  norm_plan(dtype, a.R, a.G, a.C, a.shared, false, &p);
  NORM_DISPATCH(norm_fwd_t);
}

namespace {
hipError_t norm_bwd_main(int dtype, const NormArgs& a, const NormPlan& p, hipStream_t st) {
  NORM_DISPATCH(norm_bwd_t);
}
}  // namespace

hipError_t launch_norm_bwd(int dtype, const NormArgs& a, hipStream_t st) {
  NormPlan p;
  norm_plan(dtype, a.R, a.G, a.C, a.shared, true, &p);
  if (a.R > 0) {
    const hipError_t e = norm_bwd_main(dtype, a, p, st);
    if (e != hipSuccess) return e;
  }
  if (a.dw == nullptr && a.db == nullptr) return hipSuccess;
  hipLaunchKernelGGL(col_sum_kernel, dim3((unsigned)((2 * (int64_t)p.part_cols + 15) / 16)), dim3(1024), 0, st, a.part,
                     a.R > 0 ? p.part_rows : 0, (int64_t)p.part_cols, a.dw, a.db);
  return hipGetLastError();
}

}  // namespace kda
