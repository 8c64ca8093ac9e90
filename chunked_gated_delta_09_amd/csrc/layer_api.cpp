// C ABI of the layer operators: argument checks (before any HIP call), workspace layout and launches.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include "kda_launch.h"
#include "kda_layers.h"
#include "layer_launch.h"

#define KDA_EXPORT extern "C" __attribute__((visibility("default")))

namespace {

kda_status fail(kda_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return kda::set_error(st, buf);
}

constexpr size_t kAlign = 256;
size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

#define REQUIRE(ptr, name) \
  if ((ptr) == nullptr) return fail(KDA_EINVAL, "%s is NULL", name)

// Offsets into arrays of states and tokens are 64 bits wide in the kernels; what is limited are the
// grids (one dimension of workgroups) and the 32-bit token numbers of cu_seqlens.
constexpr int64_t kMaxTokens = INT32_MAX - 64;
constexpr int64_t kMaxBlocks = (1 << 24) - 1;  // workgroups of 256: fewer than 2^32 threads
constexpr int kMaxChannels = 1 << 20;
constexpr int64_t kMaxRow = 1 << 25;
constexpr int kMaxStepRows = 65535;  // second grid dimension

kda_status hip_status(hipError_t e, const char* what) {
  return e == hipSuccess ? KDA_OK : fail(KDA_EHIP, "%s: %s", what, hipGetErrorString(e));
}

kda_status check_dtype(int dtype) {
  if (dtype != KDA_F32 && dtype != KDA_BF16) return fail(KDA_EINVAL, "unknown dtype %d", dtype);
  return KDA_OK;
}

// Rows of states that fill a lane's four are read and written 16 bytes at a time.
kda_status check_aligned(const void* p, const char* name, int NS) {
  if (NS == kda::scan_np(NS) && reinterpret_cast<uintptr_t>(p) % 16 != 0) return fail(KDA_EINVAL, "%s must be 16-byte aligned", name);
  return KDA_OK;
}

kda_status check_ws(void* ws, size_t ws_bytes, size_t need) {
  if (need == 0) return KDA_OK;
  if (ws == nullptr) return fail(KDA_EINVAL, "workspace is NULL (%zu bytes needed)", need);
  if (ws_bytes < need) return fail(KDA_EINVAL, "workspace too small: %zu bytes given, %zu needed", ws_bytes, need);
  if (reinterpret_cast<uintptr_t>(ws) % kAlign != 0) return fail(KDA_EINVAL, "workspace must be 256-byte aligned");
  return KDA_OK;
}

// A row of 0 stands for the tensor's own width.
kda_status row_of(int64_t given, int64_t width, const char* name, int64_t* row) {
  if (given != 0 && given < width)
    return fail(KDA_EINVAL, "%s_row (%lld) must be 0 or at least the width (%lld)", name, (long long)given, (long long)width);
  // the scan holds a chunk's offsets (16 rows) in 32 bits
  if (given > kMaxRow) return fail(KDA_EINVAL, "%s_row must be at most %lld, got %lld", name, (long long)kMaxRow, (long long)given);
  *row = given == 0 ? width : given;
  return KDA_OK;
}

#define TRY(expr)                          \
  do {                                     \
    const kda_status st_ = (expr);         \
    if (st_ != KDA_OK) return st_;         \
  } while (0)

struct Tokens {
  kda::Seqs sq;
  int64_t longest = 0;
};

kda_status check_tokens(int B, int T, int N, const int32_t* cu_dev, const int32_t* cu_host, bool launching, Tokens* t) {
  if (B <= 0 || N <= 0 || T < 0) return fail(KDA_EINVAL, "dims must be positive (B=%d T=%d N=%d)", B, T, N);
  if (launching && (cu_dev == nullptr) != (cu_host == nullptr))
    return fail(KDA_EINVAL, "cu_seqlens_dev and cu_seqlens_host must be both given or both NULL");
  t->sq.n = N;
  t->sq.T = T;
  t->sq.total = (int64_t)B * T;
  t->sq.cu = nullptr;
  if (t->sq.total > kMaxTokens) return fail(KDA_EINVAL, "too many tokens (%lld)", (long long)t->sq.total);
  if (cu_host != nullptr) {
    if (B != 1) return fail(KDA_EINVAL, "packed sequences (cu_seqlens given) need B = 1, got %d", B);
    if (cu_host[0] != 0) return fail(KDA_EINVAL, "cu_seqlens[0] must be 0, got %d", cu_host[0]);
    for (int n = 0; n < N; ++n) {
      if (cu_host[n + 1] < cu_host[n])
        return fail(KDA_EINVAL, "cu_seqlens must be non-decreasing (cu[%d]=%d > cu[%d]=%d)", n, cu_host[n], n + 1, cu_host[n + 1]);
      if (cu_host[n + 1] - cu_host[n] > t->longest) t->longest = cu_host[n + 1] - cu_host[n];
    }
    if (cu_host[N] != T) return fail(KDA_EINVAL, "cu_seqlens[N] (%d) must equal T (%d)", cu_host[N], T);
    t->sq.cu = cu_dev;
  } else {
    if (N != B) return fail(KDA_EINVAL, "dense batches need N == B (N=%d, B=%d)", N, B);
    t->longest = T;
  }
  return KDA_OK;
}

kda_status check_step(const char* what, int B, int T, int N, const int32_t* cu_dev, const int32_t* cu_host,
                      const int32_t* slots, int32_t S) {
  if (B <= 0 || B > kMaxStepRows) return fail(KDA_EINVAL, "%s needs 1 <= B <= %d, got %d", what, kMaxStepRows, B);
  if (T != 1 || N != B || cu_dev != nullptr || cu_host != nullptr)
    return fail(KDA_EINVAL, "%s takes one token per sequence (T = 1, N = B, no cu_seqlens)", what);
  if (S <= 0) return fail(KDA_EINVAL, "S (rows of the state) must be positive, got %d", S);
  if (slots == nullptr && S < B) return fail(KDA_EINVAL, "without slots the state needs a row for each of B = %d, got S = %d", B, S);
  return KDA_OK;
}

// ---- short convolution

kda_status conv_check(const kda_conv_dims* d, bool launching, Tokens* t, kda::ConvArgs* a) {
  if (d == nullptr) return fail(KDA_EINVAL, "dims is NULL");
  TRY(check_tokens(d->B, d->T, d->N, d->cu_seqlens_dev, d->cu_seqlens_host, launching, t));
  if (d->D <= 0 || d->D > kMaxChannels) return fail(KDA_EINVAL, "D must be in 1 .. %d, got %d", kMaxChannels, d->D);
  if (d->W < 2 || d->W > 4) return fail(KDA_EUNSUPPORTED, "W must be 2, 3 or 4, got %d", d->W);
  if (d->act != KDA_ACT_NONE && d->act != KDA_ACT_SILU) return fail(KDA_EINVAL, "act must be none or silu, got %d", d->act);
  TRY(check_dtype(d->dtype));
  *a = kda::ConvArgs{};
  TRY(row_of(d->x_row, d->D, "x", &a->x_row));
  // a run has at least 8 tokens, 64 where there are enough of them
  if (t->sq.total / 64 + d->N + (1 << 20) > kMaxBlocks) return fail(KDA_EINVAL, "too many tokens (%lld)", (long long)t->sq.total);
  a->sq = t->sq;
  a->D = d->D;
  a->W = d->W;
  a->act = d->act;
  return KDA_OK;
}

// The backward's runs do not depend on what its pointers allow, so that the workspace has one size.
size_t conv_bwd_ws(const kda_conv_dims* d, kda::ConvArgs* a) {
  a->tt = kda::conv_tile(a->sq.total, a->D, 4);
  return align_up((size_t)kda::conv_row_blocks(*a) * (d->W + 1) * d->D * sizeof(float));
}

}  // namespace

KDA_EXPORT kda_status kda_short_conv_fwd(const kda_conv_dims* dims, const void* x, const float* weight,
                                         const float* bias, const void* h0, void* y, void* final_state, void* stream) {
  Tokens t;
  kda::ConvArgs a;
  TRY(conv_check(dims, true, &t, &a));
  REQUIRE(weight, "weight");
  if (a.sq.total > 0) {
    REQUIRE(x, "x");
    REQUIRE(y, "y");
  }
  a.x = x;
  a.w = weight;
  a.wvec = reinterpret_cast<uintptr_t>(weight) % 16 == 0;
  a.bias = bias;
  a.h0 = h0;
  a.y = y;
  a.final_state = final_state;
  const void* p[4] = {x, h0, y, final_state};
  a.vec = kda::conv_vec(dims->dtype, a.D, a.x_row, p, 4);
  a.tt = kda::conv_tile(a.sq.total, a.D, a.vec);
  return hip_status(kda::launch_conv_fwd(dims->dtype, a, static_cast<hipStream_t>(stream)), "kda_short_conv_fwd");
}

KDA_EXPORT size_t kda_short_conv_bwd_workspace_bytes(const kda_conv_dims* dims) {
  Tokens t;
  kda::ConvArgs a;
  if (conv_check(dims, false, &t, &a) != KDA_OK) return 0;
  return conv_bwd_ws(dims, &a);
}

KDA_EXPORT kda_status kda_short_conv_bwd(const kda_conv_dims* dims, const void* x, const float* weight,
                                         const float* bias, const void* h0, const void* dy, const void* dfinal,
                                         void* dx, float* dweight, float* dbias, void* dh0, void* workspace,
                                         size_t ws_bytes, void* stream) {
  Tokens t;
  kda::ConvArgs a;
  TRY(conv_check(dims, true, &t, &a));
  REQUIRE(weight, "weight");
  REQUIRE(dweight, "dweight");
  if (a.sq.total > 0) {
    REQUIRE(x, "x");
    REQUIRE(dy, "dy");
    REQUIRE(dx, "dx");
  }
  TRY(check_ws(workspace, ws_bytes, conv_bwd_ws(dims, &a)));
  a.x = x;
  a.w = weight;
  a.wvec = reinterpret_cast<uintptr_t>(weight) % 16 == 0;
  a.bias = bias;
  a.h0 = h0;
  a.dy = dy;
  a.dfinal = dfinal;
  a.dx = dx;
  a.dw = dweight;
  a.db = dbias;
  a.dh0 = dh0;
  a.part = static_cast<float*>(workspace);
  const void* p[6] = {x, h0, dy, dfinal, dx, dh0};
  a.vec = kda::conv_vec(dims->dtype, a.D, a.x_row, p, 6);
  return hip_status(kda::launch_conv_bwd(dims->dtype, a, static_cast<hipStream_t>(stream)), "kda_short_conv_bwd");
}

KDA_EXPORT kda_status kda_short_conv_step(const kda_conv_dims* dims, const void* x, const float* weight,
                                          const float* bias, const int32_t* slots, int32_t S, void* state, void* y,
                                          void* stream) {
  Tokens t;
  kda::ConvArgs c;
  TRY(conv_check(dims, false, &t, &c));
  TRY(check_step("kda_short_conv_step", dims->B, dims->T, dims->N, dims->cu_seqlens_dev, dims->cu_seqlens_host, slots, S));
  REQUIRE(x, "x");
  REQUIRE(weight, "weight");
  REQUIRE(state, "state");
  REQUIRE(y, "y");
  kda::ConvStepArgs a{};
  a.B = dims->B;
  a.D = dims->D;
  a.W = dims->W;
  a.act = dims->act;
  a.slots_n = S;
  a.x_row = c.x_row;
  a.x = x;
  a.w = weight;
  a.wvec = reinterpret_cast<uintptr_t>(weight) % 16 == 0;
  a.bias = bias;
  a.slots = slots;
  a.state = state;
  a.y = y;
  return hip_status(kda::launch_conv_step(dims->dtype, a, static_cast<hipStream_t>(stream)), "kda_short_conv_step");
}

// ---- selective scan

namespace {

kda_status sscan_check(const kda_sscan_dims* d, bool launching, Tokens* t, kda::ScanArgs* a) {
  if (d == nullptr) return fail(KDA_EINVAL, "dims is NULL");
  TRY(check_tokens(d->B, d->T, d->N, d->cu_seqlens_dev, d->cu_seqlens_host, launching, t));
  if (d->D <= 0 || d->D > kMaxChannels) return fail(KDA_EINVAL, "D must be in 1 .. %d, got %d", kMaxChannels, d->D);
  if (d->NS <= 0 || d->NS > 64) return fail(KDA_EUNSUPPORTED, "NS (states per channel) must be in 1 .. 64, got %d", d->NS);
  if (d->G <= 0 || d->D % d->G != 0) return fail(KDA_EINVAL, "D (%d) must be a multiple of G (%d)", d->D, d->G);
  if (d->softplus != 0 && d->softplus != 1) return fail(KDA_EINVAL, "softplus must be 0 or 1, got %d", d->softplus);
  TRY(check_dtype(d->dtype));
  *a = kda::ScanArgs{};
  TRY(row_of(d->x_row, d->D, "x", &a->x_row));
  TRY(row_of(d->dt_row, d->D, "dt", &a->dt_row));
  TRY(row_of(d->z_row, d->D, "z", &a->z_row));
  TRY(row_of(d->b_row, (int64_t)d->G * d->NS, "b", &a->b_row));
  TRY(row_of(d->c_row, (int64_t)d->G * d->NS, "c", &a->c_row));
  a->sq = t->sq;
  a->D = d->D;
  a->N = d->NS;
  a->G = d->G;
  a->softplus = d->softplus;
  const int64_t cols = (int64_t)d->G * kda::scan_tiles(d->D, d->NS, d->G);
  // a local segment has at least 16 tokens, or is a sequence of its own
  if ((t->sq.total / 16 + d->N) * cols > kMaxBlocks)
    return fail(KDA_EINVAL, "too many channel tiles (%lld tokens x %lld)", (long long)t->sq.total, (long long)cols);
  if (t->sq.total * d->G * kda::scan_np(d->NS) / 512 + 2 * (int64_t)d->D > kMaxBlocks) return fail(KDA_EINVAL, "too many tokens for G * NS = %d", d->G * d->NS);
  return KDA_OK;
}

struct ScanLayout {
  int seg = 0, lseg = 0;
  int64_t nseg = 0, nloc = 0, chunks = 0;
  bool split = false;
  size_t segoff = 0, loff = 0, choff = 0, seg_dt = 0, seg_state = 0, part_bc = 0, part_a = 0, part_d = 0, total = 0;
};

ScanLayout scan_layout(const kda_sscan_dims* d, const Tokens& t, bool bwd) {
  ScanLayout l;
  kda::scan_seg(t.sq, t.longest, d->D, d->NS, d->G, bwd, &l.seg, &l.lseg);
  l.split = t.longest > l.seg;
  for (int n = 0; n < d->N; ++n) {
    const int64_t len = d->cu_seqlens_host != nullptr ? d->cu_seqlens_host[n + 1] - d->cu_seqlens_host[n] : d->T;
    l.nseg += len > 0 ? (len + l.seg - 1) / l.seg : 1;
    l.nloc += len > 0 ? (len + l.lseg - 1) / l.lseg : 1;
    l.chunks += (len + kda::kScanChunk - 1) / kda::kScanChunk;
  }
  const size_t NP = kda::scan_np(d->NS), D = d->D;
  size_t o = 0;
  if (d->cu_seqlens_host != nullptr && d->N > kda::kScanLanes) {
    l.segoff = o; o = align_up(o + sizeof(int32_t) * (d->N + 1));
    l.loff = o; o = align_up(o + sizeof(int32_t) * (d->N + 1));
    l.choff = o; o = align_up(o + sizeof(int32_t) * (d->N + 1));
  }
  if (l.split) {
    l.seg_dt = o; o = align_up(o + (size_t)l.nloc * D * sizeof(float));
    l.seg_state = o; o = align_up(o + (size_t)l.nloc * D * NP * sizeof(float));
  }
  if (bwd) {
    l.part_bc = o; o = align_up(o + (size_t)kda::scan_tiles(d->D, d->NS, d->G) * t.sq.total * d->G * 2 * NP * sizeof(float));
    l.part_a = o; o = align_up(o + (size_t)l.nseg * D * NP * sizeof(float));
    l.part_d = o; o = align_up(o + (size_t)l.nseg * 2 * D * sizeof(float));
  }
  l.total = o;
  return l;
}

void scan_use(const ScanLayout& l, void* workspace, kda::ScanArgs* a) {
  char* ws = static_cast<char*>(workspace);
  a->seg = l.seg;
  a->nseg = l.nseg;
  a->split = l.split;
  a->lseg = l.lseg;
  a->nloc = l.nloc;
  a->loff = reinterpret_cast<int32_t*>(ws + l.loff);
  a->segoff = reinterpret_cast<int32_t*>(ws + l.segoff);
  a->choff = reinterpret_cast<int32_t*>(ws + l.choff);
  a->seg_dt = reinterpret_cast<float*>(ws + l.seg_dt);
  a->seg_state = reinterpret_cast<float*>(ws + l.seg_state);
  a->part_bc = reinterpret_cast<float*>(ws + l.part_bc);
  a->part_a = reinterpret_cast<float*>(ws + l.part_a);
  a->part_d = reinterpret_cast<float*>(ws + l.part_d);
}

// Four-element loads: every row of these tensors, and a group's first channel, on a multiple of four.
int scan_vec(const kda::ScanArgs& a, int dtype, const void* const* ptrs, int np) {
  const int es = dtype == KDA_F32 ? 4 : 2;
  bool ok = (a.D / a.G) % 4 == 0 && a.x_row % 4 == 0 && a.dt_row % 4 == 0 && (a.z == nullptr || a.z_row % 4 == 0);
  for (int i = 0; i < np; ++i) ok = ok && reinterpret_cast<uintptr_t>(ptrs[i]) % (4 * es) == 0;
  return ok;
}

kda_status scan_tables(const kda_sscan_dims* d, const ScanLayout& l, void* workspace, const kda::ScanArgs& a, hipStream_t st) {
  if (d->cu_seqlens_host == nullptr || d->N <= kda::kScanLanes) return KDA_OK;
  char* ws = static_cast<char*>(workspace);
  return hip_status(kda::launch_scan_tables(a.sq, l.seg, l.lseg, reinterpret_cast<int32_t*>(ws + l.segoff),
                                            reinterpret_cast<int32_t*>(ws + l.loff),
                                            reinterpret_cast<int32_t*>(ws + l.choff), st), "segment table");
}

}  // namespace

KDA_EXPORT int64_t kda_sscan_num_chunks(const kda_sscan_dims* dims) {
  Tokens t;
  kda::ScanArgs a;
  if (sscan_check(dims, false, &t, &a) != KDA_OK) return -1;
  return scan_layout(dims, t, false).chunks;
}

KDA_EXPORT size_t kda_sscan_fwd_workspace_bytes(const kda_sscan_dims* dims) {
  Tokens t;
  kda::ScanArgs a;
  if (sscan_check(dims, false, &t, &a) != KDA_OK) return 0;
  return scan_layout(dims, t, false).total;
}

KDA_EXPORT size_t kda_sscan_bwd_workspace_bytes(const kda_sscan_dims* dims) {
  Tokens t;
  kda::ScanArgs a;
  if (sscan_check(dims, false, &t, &a) != KDA_OK) return 0;
  return scan_layout(dims, t, true).total;
}

KDA_EXPORT kda_status kda_sscan_fwd(const kda_sscan_dims* dims, const void* x, const void* dt, const float* A,
                                    const void* Bm, const void* Cm, const float* skip, const void* z,
                                    const float* dt_bias, const float* h0, void* y, float* final_state, float* states,
                                    void* workspace, size_t ws_bytes, void* stream) {
  Tokens t;
  kda::ScanArgs a;
  TRY(sscan_check(dims, true, &t, &a));
  REQUIRE(A, "A");
  if (a.sq.total > 0) {
    REQUIRE(x, "x");
    REQUIRE(dt, "dt");
    REQUIRE(Bm, "B");
    REQUIRE(Cm, "C");
    REQUIRE(y, "y");
  }
  TRY(check_aligned(A, "A", dims->NS));
  TRY(check_aligned(h0, "h0", dims->NS));
  TRY(check_aligned(final_state, "final_state", dims->NS));
  TRY(check_aligned(states, "states", dims->NS));
  const ScanLayout l = scan_layout(dims, t, false);
  TRY(check_ws(workspace, ws_bytes, l.total));
  a.x = x;
  a.dt = dt;
  a.z = z;
  a.B = Bm;
  a.C = Cm;
  a.A = A;
  a.skip = skip;
  a.dt_bias = dt_bias;
  a.h0 = h0;
  a.y = y;
  a.final_state = final_state;
  a.states = states;
  scan_use(l, workspace, &a);
  const void* p[4] = {x, dt, z, y};
  a.vec = scan_vec(a, dims->dtype, p, 4);
  hipStream_t st = static_cast<hipStream_t>(stream);
  TRY(scan_tables(dims, l, workspace, a, st));
  return hip_status(kda::launch_sscan_fwd(dims->dtype, a, st), "kda_sscan_fwd");
}

KDA_EXPORT kda_status kda_sscan_bwd(const kda_sscan_dims* dims, const void* x, const void* dt, const float* A,
                                    const void* Bm, const void* Cm, const float* skip, const void* z,
                                    const float* dt_bias, const float* states, const void* dy, const float* dfinal,
                                    void* dx, void* ddt, float* dA, void* dB, void* dC, float* dskip, void* dz,
                                    float* ddt_bias, float* dh0, void* workspace, size_t ws_bytes, void* stream) {
  Tokens t;
  kda::ScanArgs a;
  TRY(sscan_check(dims, true, &t, &a));
  REQUIRE(A, "A");
  REQUIRE(dA, "dA");
  if (a.sq.total > 0) {
    REQUIRE(x, "x");
    REQUIRE(dt, "dt");
    REQUIRE(Bm, "B");
    REQUIRE(Cm, "C");
    REQUIRE(states, "states");
    REQUIRE(dy, "dy");
    REQUIRE(dx, "dx");
    REQUIRE(ddt, "ddt");
    REQUIRE(dB, "dB");
    REQUIRE(dC, "dC");
  }
  if (dz != nullptr) REQUIRE(z, "z (needed for dz)");
  if (dskip != nullptr) REQUIRE(skip, "skip (needed for dskip)");
  TRY(check_aligned(A, "A", dims->NS));
  TRY(check_aligned(states, "states", dims->NS));
  TRY(check_aligned(dfinal, "dfinal", dims->NS));
  TRY(check_aligned(dh0, "dh0", dims->NS));
  const ScanLayout l = scan_layout(dims, t, true);
  TRY(check_ws(workspace, ws_bytes, l.total));
  a.x = x;
  a.dt = dt;
  a.z = z;
  a.B = Bm;
  a.C = Cm;
  a.A = A;
  a.skip = skip;
  a.dt_bias = dt_bias;
  a.states = const_cast<float*>(states);
  a.dy = dy;
  a.dfinal = dfinal;
  a.dx = dx;
  a.ddt = ddt;
  a.dA = dA;
  a.dB = dB;
  a.dC = dC;
  a.dskip = dskip;
  a.dz = dz;
  a.ddt_bias = ddt_bias;
  a.dh0 = dh0;
  scan_use(l, workspace, &a);
  const void* p[7] = {x, dt, z, dy, dx, ddt, dz};
  a.vec = scan_vec(a, dims->dtype, p, 7);
  const uintptr_t bc = reinterpret_cast<uintptr_t>(dB) | reinterpret_cast<uintptr_t>(dC);
  a.bcvec = a.N % 4 == 0 && bc % (dims->dtype == KDA_F32 ? 16 : 8) == 0;
  hipStream_t st = static_cast<hipStream_t>(stream);
  TRY(scan_tables(dims, l, workspace, a, st));
  return hip_status(kda::launch_sscan_bwd(dims->dtype, a, st), "kda_sscan_bwd");
}

KDA_EXPORT kda_status kda_sscan_step(const kda_sscan_dims* dims, const void* x, const void* dt, const float* A,
                                     const void* Bm, const void* Cm, const float* skip, const void* z,
                                     const float* dt_bias, const int32_t* slots, int32_t S, float* state, void* y,
                                     void* stream) {
  Tokens t;
  kda::ScanArgs c;
  TRY(sscan_check(dims, false, &t, &c));
  TRY(check_step("kda_sscan_step", dims->B, dims->T, dims->N, dims->cu_seqlens_dev, dims->cu_seqlens_host, slots, S));
  REQUIRE(x, "x");
  REQUIRE(dt, "dt");
  REQUIRE(A, "A");
  REQUIRE(Bm, "B");
  REQUIRE(Cm, "C");
  REQUIRE(state, "state");
  REQUIRE(y, "y");
  TRY(check_aligned(A, "A", dims->NS));
  TRY(check_aligned(state, "state", dims->NS));
  kda::ScanStepArgs a{};
  a.B = dims->B;
  a.D = dims->D;
  a.N = dims->NS;
  a.G = dims->G;
  a.softplus = dims->softplus;
  a.slots_n = S;
  a.x_row = c.x_row;
  a.dt_row = c.dt_row;
  a.z_row = c.z_row;
  a.b_row = c.b_row;
  a.c_row = c.c_row;
  a.x = x;
  a.dt = dt;
  a.z = z;
  a.Bm = Bm;
  a.Cm = Cm;
  a.A = A;
  a.skip = skip;
  a.dt_bias = dt_bias;
  a.slots = slots;
  a.state = state;
  a.y = y;
  return hip_status(kda::launch_sscan_step(dims->dtype, a, static_cast<hipStream_t>(stream)), "kda_sscan_step");
}

// ---- group norm

namespace {

kda_status norm_check(const kda_norm_dims* d, kda::NormArgs* a) {
  if (d == nullptr) return fail(KDA_EINVAL, "dims is NULL");
  if (d->R < 0 || d->G <= 0 || d->C <= 0) return fail(KDA_EINVAL, "dims must be positive (R=%lld G=%d C=%d)", (long long)d->R, d->G, d->C);
  if (d->C > 8192) return fail(KDA_EUNSUPPORTED, "C (channels of a group) must be at most 8192, got %d", d->C);
  if ((int64_t)d->G * d->C > kMaxChannels) return fail(KDA_EINVAL, "G * C must be at most %d, got %lld", kMaxChannels, (long long)d->G * d->C);
  if (d->R > kMaxTokens || d->R * d->G > kMaxTokens) return fail(KDA_EINVAL, "too many groups (R=%lld G=%d)", (long long)d->R, d->G);
  if (d->center != 0 && d->center != 1) return fail(KDA_EINVAL, "center must be 0 or 1, got %d", d->center);
  if (d->shared != 0 && d->shared != 1) return fail(KDA_EINVAL, "shared must be 0 or 1, got %d", d->shared);
  if (d->act < KDA_ACT_NONE || d->act > KDA_ACT_SIGMOID) return fail(KDA_EINVAL, "unknown act %d", d->act);
  if (!(d->eps > 0.f) || !std::isfinite(d->eps)) return fail(KDA_EINVAL, "eps must be positive and finite");
  TRY(check_dtype(d->dtype));
  *a = kda::NormArgs{};
  TRY(row_of(d->x_row, (int64_t)d->G * d->C, "x", &a->x_row));
  TRY(row_of(d->gate_row, (int64_t)d->G * d->C, "gate", &a->gate_row));
  a->R = d->R;
  a->G = d->G;
  a->C = d->C;
  a->center = d->center;
  a->act = d->act;
  a->shared = d->shared;
  a->eps = d->eps;
  return KDA_OK;
}

int norm_vec(const kda::NormArgs& a, int dtype, const void* const* ptrs, int np) {
  const int es = dtype == KDA_F32 ? 4 : 2, vec = 16 / es;
  bool ok = a.C % vec == 0 && a.x_row % vec == 0 && (a.gate == nullptr || a.gate_row % vec == 0);
  for (int i = 0; i < np; ++i) ok = ok && reinterpret_cast<uintptr_t>(ptrs[i]) % 16 == 0;
  return ok;
}

// Weight and bias allow four-element loads: a group's first channel is on a multiple of four.
int norm_wvec(const kda::NormArgs& a, const float* w, const float* b) {
  return a.C % 4 == 0 && reinterpret_cast<uintptr_t>(w) % 16 == 0 && reinterpret_cast<uintptr_t>(b) % 16 == 0;
}

size_t norm_ws(const kda_norm_dims* d) {
  kda::NormPlan p;
  kda::norm_plan(d->dtype, d->R, d->G, d->C, d->shared, true, &p);
  return align_up((size_t)p.part_rows * 2 * p.part_cols * sizeof(float));
}

}  // namespace

KDA_EXPORT kda_status kda_group_norm_fwd(const kda_norm_dims* dims, const void* x, const float* weight,
                                         const float* bias, const void* gate, void* y, void* stream) {
  kda::NormArgs a;
  TRY(norm_check(dims, &a));
  if (a.R > 0) {
    REQUIRE(x, "x");
    REQUIRE(y, "y");
  }
  a.x = x;
  a.w = weight;
  a.bias = bias;
  a.gate = gate;
  a.y = y;
  const void* p[3] = {x, gate, y};
  a.vec = norm_vec(a, dims->dtype, p, 3);
  a.wvec = norm_wvec(a, weight, bias);
  return hip_status(kda::launch_norm_fwd(dims->dtype, a, static_cast<hipStream_t>(stream)), "kda_group_norm_fwd");
}

KDA_EXPORT size_t kda_group_norm_bwd_workspace_bytes(const kda_norm_dims* dims) {
  kda::NormArgs a;
  if (norm_check(dims, &a) != KDA_OK) return 0;
  return norm_ws(dims);
}

KDA_EXPORT kda_status kda_group_norm_bwd(const kda_norm_dims* dims, const void* x, const float* weight,
                                         const float* bias, const void* gate, const void* dy, void* dx,
                                         float* dweight, float* dbias, void* dgate, void* workspace, size_t ws_bytes,
                                         void* stream) {
  kda::NormArgs a;
  TRY(norm_check(dims, &a));
  if (a.R > 0) {
    REQUIRE(x, "x");
    REQUIRE(dy, "dy");
    REQUIRE(dx, "dx");
    if (gate != nullptr) REQUIRE(dgate, "dgate");
  }
  const bool sums = dweight != nullptr || dbias != nullptr;
  if (sums) TRY(check_ws(workspace, ws_bytes, norm_ws(dims)));
  a.x = x;
  a.w = weight;
  a.bias = bias;
  a.gate = gate;
  a.dy = dy;
  a.dx = dx;
  a.dw = dweight;
  a.db = dbias;
  a.dgate = dgate;
  a.part = sums ? static_cast<float*>(workspace) : nullptr;
  const void* p[5] = {x, gate, dy, dx, dgate};
  a.vec = norm_vec(a, dims->dtype, p, 5);
  a.wvec = norm_wvec(a, weight, bias);
  return hip_status(kda::launch_norm_bwd(dims->dtype, a, static_cast<hipStream_t>(stream)), "kda_group_norm_bwd");
}

// ---- KDA token step

KDA_EXPORT kda_status kda_step(const kda_dims* dims, const void* q, const void* k, const void* v, const float* g,
                               const float* beta, const int32_t* slots, int32_t S, float* state, void* o,
                               void* stream) {
  if (dims == nullptr) return fail(KDA_EINVAL, "dims is NULL");
  TRY(check_step("kda_step", dims->B, dims->T, dims->N, dims->cu_seqlens_dev, dims->cu_seqlens_host, slots, S));
  if (dims->H <= 0 || dims->HV <= 0 || dims->K <= 0 || dims->V <= 0)
    return fail(KDA_EINVAL, "dims must be positive (H=%d HV=%d K=%d V=%d)", dims->H, dims->HV, dims->K, dims->V);
  if (dims->HV % dims->H != 0) return fail(KDA_EINVAL, "HV (%d) must be a multiple of H (%d)", dims->HV, dims->H);
  if (dims->K > 256 || dims->V > 256) return fail(KDA_EUNSUPPORTED, "K and V must be at most 256, got %d and %d", dims->K, dims->V);
  if (dims->HV > 1 << 20) return fail(KDA_EINVAL, "too many value heads (%d)", dims->HV);
  if (dims->beta_logits != 0 && dims->beta_logits != 1)
    return fail(KDA_EINVAL, "beta_logits must be 0 or 1, got %d", dims->beta_logits);
  if (!std::isfinite(dims->scale)) return fail(KDA_EINVAL, "scale must be finite");
  TRY(check_dtype(dims->dtype));
  REQUIRE(q, "q");
  REQUIRE(k, "k");
  REQUIRE(v, "v");
  REQUIRE(g, "g");
  REQUIRE(beta, "beta");
  REQUIRE(state, "state");
  REQUIRE(o, "o");
  kda::KdaStepArgs a{};
  a.B = dims->B;
  a.H = dims->H;
  a.HV = dims->HV;
  a.K = dims->K;
  a.V = dims->V;
  a.slots_n = S;
  a.beta_logits = dims->beta_logits;
  a.scale = dims->scale;
  a.q = q;
  a.k = k;
  a.v = v;
  a.g = g;
  a.beta = beta;
  a.slots = slots;
  a.state = state;
  a.o = o;
  return hip_status(kda::launch_kda_step(dims->dtype, a, static_cast<hipStream_t>(stream)), "kda_step");
}
