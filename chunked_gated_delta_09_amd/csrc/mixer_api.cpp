// C ABI of the token mixers: argument checks (before any HIP call), workspace layout and launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "api_checks.h"
#include "kda_mixers.h"
#include "mixer_launch.h"

namespace {

bool aligned(std::initializer_list<const void*> ptrs, size_t n) {
  uintptr_t all = 0;
  for (const void* p : ptrs) all |= reinterpret_cast<uintptr_t>(p);
  return all % n == 0;
}

// Rows of the mixers' tensors: a tile's offsets are held in 32 bits.
constexpr int64_t kMaxTileRow = 1 << 23;
kda_status tile_row(int64_t given, int64_t width, const char* name, int64_t* row) {
  TRY(row_of(given, width, name, row));
  if (*row > kMaxTileRow) return fail(KDA_EINVAL, "%s_row must be at most %lld, got %lld", name, (long long)kMaxTileRow, (long long)*row);
  return KDA_OK;
}

// Runs of `seg` tokens over all sequences, each without its first `skip` tokens and with at least one run.
int64_t count_runs(const int32_t* cu, int N, int T, int64_t seg, int64_t skip) {
  auto runs = [&](int64_t len) { return len - skip > seg ? (len - skip - 1) / seg + 1 : 1; };
  if (cu == nullptr) return N * runs(T);
  int64_t n = 0;
  for (int i = 0; i < N; ++i) n += runs((int64_t)cu[i + 1] - cu[i]);
  return n;
}

// ---- linear attention

struct LinPlan {
  Tokens t;
  int seg = 0;
  int64_t nseg = 0;
  bool split = false;
  int64_t q_row = 0, k_row = 0, v_row = 0;
  int tile_k = 0, tile_v = 0;
  int slice = 0;  // elements of a state that a workgroup of the scan carries
  int tiles = 0;  // of the gradients of q and k
};

kda_status lin_check(const kda_lattn_dims* d, bool launching, LinPlan* p) {
  if (d == nullptr) return fail(KDA_EINVAL, "dims is NULL");
  TRY(check_tokens(d->B, d->T, d->N, d->cu_seqlens_dev, d->cu_seqlens_host, launching, &p->t));
  if (d->H <= 0 || d->HV <= 0 || d->K <= 0 || d->V <= 0)
    return fail(KDA_EINVAL, "dims must be positive (H=%d HV=%d K=%d V=%d)", d->H, d->HV, d->K, d->V);
  if (d->HV % d->H != 0) return fail(KDA_EINVAL, "HV (%d) must be a multiple of H (%d)", d->HV, d->H);
  if (d->K > 256 || d->V > 256) return fail(KDA_EUNSUPPORTED, "K and V must be at most 256, got %d and %d", d->K, d->V);
  if (d->HV > 1 << 16) return fail(KDA_EINVAL, "too many value heads (%d)", d->HV);
  if (d->g_const != 0 && d->g_const != 1) return fail(KDA_EINVAL, "g_const must be 0 or 1, got %d", d->g_const);
  if (!std::isfinite(d->scale)) return fail(KDA_EINVAL, "scale must be finite");
  TRY(check_dtype(d->dtype));
  TRY(tile_row(d->q_row, (int64_t)d->H * d->K, "q", &p->q_row));
  TRY(tile_row(d->k_row, (int64_t)d->H * d->K, "k", &p->k_row));
  TRY(tile_row(d->v_row, (int64_t)d->HV * d->V, "v", &p->v_row));
  // sequences of packed batches count by their tokens
  const int64_t longest = std::max<int64_t>(p->t.longest, 1), like = std::max<int64_t>(1, p->t.sq.total / longest);
  const kda::LinCut cut = kda::lin_cut(d->dtype, longest, like * d->HV, d->K, d->V);
  p->seg = cut.seg;
  p->tile_k = cut.tile_k;
  p->tile_v = cut.tile_v;
  p->nseg = count_runs(d->cu_seqlens_host, d->N, d->T, p->seg, 0);
  p->split = p->t.longest > p->seg;
  p->slice = kda::lin_scan_slice((longest + p->seg - 1) / p->seg);
  p->tiles = (d->K + p->tile_k - 1) / p->tile_k;
  // rows of the outputs, in tiles whose offsets are held in 32 bits
  if ((int64_t)d->HV * std::max(d->K, d->V) > kMaxTileRow)
    return fail(KDA_EINVAL, "HV times K or V must be at most %lld", (long long)kMaxTileRow);
  return KDA_OK;
}

// The grids of a call over whole sequences: its walks' workgroups, counted by 256 threads (four a column of the tile), and
// with `scan` the segments' scan's.
kda_status lin_grids(const kda_lattn_dims* d, const LinPlan& p, bool bwd, bool scan) {
  const int64_t cols_v = (d->V + p.tile_v - 1) / p.tile_v * (p.tile_v / 64), cols_k = p.tiles * (p.tile_k / 64);
  const int64_t cols = bwd ? std::max(cols_k, cols_v) : cols_v, slices = scan ? kda::lin_scan_slices((int64_t)d->K * d->V, p.slice) : 0;
  if (p.nseg * d->HV * cols > kMaxBlocks || (int64_t)d->N * d->HV * slices > kMaxBlocks)
    return fail(KDA_EINVAL, "too many segments (%lld of %d sequences and %d heads)", (long long)p.nseg, d->N, d->HV);
  return KDA_OK;
}

struct LinLayout {
  size_t states = 0, decay = 0, dotq = 0, dotk = 0, dots = 0, part = 0, dq = 0, dk = 0, total = 0;
};

LinLayout lin_layout(const kda_lattn_dims* d, const LinPlan& p, bool bwd) {
  LinLayout l;
  const size_t KV = (size_t)d->K * d->V * d->HV * sizeof(float), f = sizeof(float);
  size_t o = 0;
  if (p.split) {
    // forward: used where the caller keeps no states
    l.states = o; o = align_up(o + (bwd ? p.nseg : p.nseg + d->N) * KV);
    l.decay = o; o = align_up(o + (size_t)p.nseg * d->HV * f);
  }
  if (bwd) {
    const size_t rows = (size_t)p.t.sq.total * d->HV;
    l.dotq = o; o = align_up(o + p.tiles * rows * f);
    l.dotk = o; o = align_up(o + p.tiles * rows * f);
    l.dots = o; o = align_up(o + (size_t)kda::lin_scan_slices((int64_t)d->K * d->V, p.slice) * p.nseg * d->HV * f);
    if (d->g_const) { l.part = o; o = align_up(o + (size_t)p.nseg * d->HV * sizeof(double)); }
    if (d->HV != d->H) {
      // dq's heads are summed before dk's are formed: kernels of one stream follow each other
      l.dq = l.dk = o; o = align_up(o + rows * d->K * f);
    }
  }
  l.total = o;
  return l;
}

kda::LinArgs lin_args(const kda_lattn_dims* d, const LinPlan& p, const float* g) {
  kda::LinArgs a{};
  a.sq = p.t.sq;
  a.seg = p.seg;
  a.nseg = p.nseg;
  a.HV = d->HV;
  a.rep = d->HV / d->H;
  a.g = g;
  a.g_const = d->g_const;
  a.scale = d->scale;
  return a;
}

struct Rows {
  const void* p;
  int64_t row;
  int qk;
};
// The rows of the three places, the output and the rows that it is multiplied with.
void lin_rows(kda::LinArgs* a, int dtype, int P, int R, const Rows& x, const Rows& y, const Rows& z, void* out = nullptr,
              int out_f32 = 0, const Rows& w = Rows{nullptr, 0, 0}, float* dot = nullptr) {
  a->P = P;
  a->R = R;
  a->x = x.p;
  a->y = y.p;
  a->z = z.p;
  a->x_row = x.row;
  a->y_row = y.row;
  a->z_row = z.row;
  a->x_qk = x.qk;
  a->y_qk = y.qk;
  a->z_qk = z.qk;
  a->out = out;
  a->out_f32 = out_f32;
  a->w = w.p;
  a->w_row = w.row;
  a->w_qk = w.qk;
  a->dot = dot;
  const int ev = dtype == KDA_F32 ? 4 : 8;
  a->vec = P % ev == 0 && R % ev == 0 && x.row % ev == 0 && y.row % ev == 0 && z.row % ev == 0 && w.row % ev == 0 &&
           aligned({x.p, y.p, z.p, w.p, out}, 16);
}

}  // namespace

KDA_EXPORT int64_t kda_lattn_num_states(const kda_lattn_dims* dims) {
  LinPlan p;
  if (lin_check(dims, false, &p) != KDA_OK || lin_grids(dims, p, true, p.split) != KDA_OK) return -1;
  return p.nseg + dims->N;
}

KDA_EXPORT size_t kda_lattn_fwd_workspace_bytes(const kda_lattn_dims* dims) {
  LinPlan p;
  if (lin_check(dims, false, &p) != KDA_OK || lin_grids(dims, p, false, p.split) != KDA_OK) return 0;
  return lin_layout(dims, p, false).total;
}

KDA_EXPORT size_t kda_lattn_bwd_workspace_bytes(const kda_lattn_dims* dims) {
  LinPlan p;
  if (lin_check(dims, false, &p) != KDA_OK || lin_grids(dims, p, true, p.split) != KDA_OK) return 0;
  return lin_layout(dims, p, true).total;
}

KDA_EXPORT kda_status kda_lattn_fwd(const kda_lattn_dims* dims, const void* q, const void* k, const void* v,
                                    const float* g, const float* h0, void* o, float* final_state, float* states,
                                    void* workspace, size_t ws_bytes, void* stream) {
  LinPlan p;
  TRY(lin_check(dims, true, &p));
  TRY(lin_grids(dims, p, false, p.split));
  if (p.t.sq.total > 0) {
    REQUIRE(q, "q");
    REQUIRE(k, "k");
    REQUIRE(v, "v");
    REQUIRE(g, "g");
    REQUIRE(o, "o");
  }
  const LinLayout l = lin_layout(dims, p, false);
  TRY(check_ws(workspace, ws_bytes, l.total));
  hipStream_t st = static_cast<hipStream_t>(stream);
  const int dt = dims->dtype, K = dims->K, V = dims->V;
  const Rows rq{q, p.q_row, 1}, rk{k, p.k_row, 1}, rv{v, p.v_row, 0};
  char* ws = static_cast<char*>(workspace);
  kda::LinArgs a = lin_args(dims, p, g);
  a.s_p = V;
  a.s_r = 1;
  a.tile = p.tile_v;
  lin_rows(&a, dt, K, V, rq, rk, rv, o);
  if (p.split) {
    float* all = states != nullptr ? states : reinterpret_cast<float*>(ws + l.states);
    kda::LinArgs b = a;
    b.fin = all;
    b.fin_mode = kda::kStateStart;
    b.seg_decay = reinterpret_cast<float*>(ws + l.decay);
    TRY(hip_status(kda::launch_lin_walk(dt, kda::kLinState, b, st), "kda_lattn_fwd"));
    kda::LinScanArgs s{};
    s.sq = p.t.sq;
    s.seg = p.seg;
    s.nseg = p.nseg;
    s.HV = dims->HV;
    s.KV = (int64_t)K * V;
    s.slice = p.slice;
    s.seg_decay = b.seg_decay;
    s.first = h0;
    s.states = all;
    s.last = final_state;
    s.local = 1;
    TRY(hip_status(kda::launch_lin_scan(s, false, st), "kda_lattn_fwd"));
    a.s0 = all;
    a.s0_mode = kda::kStateStart;
  } else {
    a.s0 = h0;
    a.s0_mode = h0 != nullptr ? kda::kStateSeq : kda::kStateNone;
    a.fin = final_state;
    a.fin_mode = kda::kStateSeq;
    a.fin2 = states;
    a.fin2_mode = kda::kStateEnd;
    a.copy0 = states;
  }
  const int mode = a.fin != nullptr || a.fin2 != nullptr ? kda::kLinOutFin : kda::kLinOut;
  return hip_status(kda::launch_lin_walk(dt, mode, a, st), "kda_lattn_fwd");
}

KDA_EXPORT kda_status kda_lattn_bwd(const kda_lattn_dims* dims, const void* q, const void* k, const void* v,
                                    const float* g, const float* states, const void* dout, const float* dfinal,
                                    void* dq, void* dk, void* dv, float* dg, float* dh0, void* workspace,
                                    size_t ws_bytes, void* stream) {
  LinPlan p;
  TRY(lin_check(dims, true, &p));
  const bool ends = p.split || dfinal != nullptr;  // some segment has a gradient at its end
  TRY(lin_grids(dims, p, true, ends));
  REQUIRE(states, "states");
  if (p.t.sq.total > 0 || dims->g_const) REQUIRE(dg, "dg");
  if (p.t.sq.total > 0) {
    REQUIRE(q, "q");
    REQUIRE(k, "k");
    REQUIRE(v, "v");
    REQUIRE(g, "g");
    REQUIRE(dout, "do");
    REQUIRE(dq, "dq");
    REQUIRE(dk, "dk");
    REQUIRE(dv, "dv");
  }
  const LinLayout l = lin_layout(dims, p, true);
  TRY(check_ws(workspace, ws_bytes, l.total));
  hipStream_t st = static_cast<hipStream_t>(stream);
  const int dt = dims->dtype, K = dims->K, V = dims->V, rep = dims->HV / dims->H;
  const Rows rq{q, p.q_row, 1}, rk{k, p.k_row, 1}, rv{v, p.v_row, 0}, rd{dout, (int64_t)dims->HV * V, 0}, none{nullptr, 0, 0};
  char* ws = static_cast<char*>(workspace);
  float *dotq = reinterpret_cast<float*>(ws + l.dotq), *dotk = reinterpret_cast<float*>(ws + l.dotk),
        *dots = reinterpret_cast<float*>(ws + l.dots), *rev = reinterpret_cast<float*>(ws + l.states);
  float *dqs = reinterpret_cast<float*>(ws + l.dq), *dks = reinterpret_cast<float*>(ws + l.dk);

  kda::LinArgs a = lin_args(dims, p, g);
  a.s_p = 1;
  a.s_r = V;
  a.tile = p.tile_k;
  a.s0 = states;
  a.s0_mode = kda::kStateStart;
  lin_rows(&a, dt, V, K, rd, rv, rk, rep > 1 ? dqs : dq, rep > 1, rq, dotq);
  TRY(hip_status(kda::launch_lin_walk(dt, kda::kLinDot, a, st), "kda_lattn_bwd"));
  if (rep > 1) TRY(hip_status(kda::launch_group_sum(dt, dqs, dq, p.t.sq.total * dims->H, rep, K, st), "kda_lattn_bwd"));

  kda::LinArgs b = lin_args(dims, p, g);
  if (p.split) {
    b.s_p = V;
    b.s_r = 1;
    b.tile = p.tile_v;
    lin_rows(&b, dt, K, V, none, rq, rd);
    b.fin = rev;
    b.fin_mode = kda::kStateSeg;
    b.seg_decay = reinterpret_cast<float*>(ws + l.decay);
    TRY(hip_status(kda::launch_lin_walk(dt, kda::kLinStateRev, b, st), "kda_lattn_bwd"));
  }
  if (ends) {
    kda::LinScanArgs s{};
    s.sq = p.t.sq;
    s.seg = p.seg;
    s.nseg = p.nseg;
    s.HV = dims->HV;
    s.KV = (int64_t)K * V;
    s.slice = p.slice;
    s.seg_decay = b.seg_decay;
    s.first = dfinal;
    s.states = rev;
    s.last = dh0;
    s.fwd = states;
    s.dot = dots;
    s.local = p.split;
    TRY(hip_status(kda::launch_lin_scan(s, true, st), "kda_lattn_bwd"));
  }
  kda::LinArgs c = lin_args(dims, p, g);
  c.s0 = p.split ? rev : dfinal;
  c.s0_mode = p.split ? kda::kStateSeg : dfinal != nullptr ? kda::kStateSeq : kda::kStateNone;
  kda::LinArgs e = c;
  c.s_p = 1;
  c.s_r = V;
  c.tile = p.tile_k;
  c.fin = p.split ? nullptr : dh0;
  c.fin_mode = kda::kStateSeq;
  lin_rows(&c, dt, V, K, rv, rd, rq, rep > 1 ? dks : dk, rep > 1, rk, dotk);
  TRY(hip_status(kda::launch_lin_walk(dt, kda::kLinDotRev, c, st), "kda_lattn_bwd"));
  if (rep > 1) TRY(hip_status(kda::launch_group_sum(dt, dks, dk, p.t.sq.total * dims->H, rep, K, st), "kda_lattn_bwd"));
  e.s_p = V;
  e.s_r = 1;
  e.tile = p.tile_v;
  lin_rows(&e, dt, K, V, rk, rq, rd, dv);
  TRY(hip_status(kda::launch_lin_walk(dt, kda::kLinOutRev, e, st), "kda_lattn_bwd"));
  kda::LinGateArgs f{};
  f.sq = p.t.sq;
  f.seg = p.seg;
  f.nseg = p.nseg;
  f.HV = dims->HV;
  f.qtiles = f.ktiles = p.tiles;
  f.slices = ends ? kda::lin_scan_slices((int64_t)K * V, p.slice) : 0;
  f.dotq = dotq;
  f.dotk = dotk;
  f.dots = dots;
  f.dg = dg;
  f.part = dims->g_const ? reinterpret_cast<double*>(ws + l.part) : nullptr;
  return hip_status(kda::launch_lin_gate(f, st), "kda_lattn_bwd");
}

KDA_EXPORT kda_status kda_lattn_step(const kda_lattn_dims* dims, const void* q, const void* k, const void* v,
                                     const float* g, const int32_t* slots, int32_t S, float* state, void* o,
                                     void* stream) {
  LinPlan p;
  TRY(lin_check(dims, false, &p));
  TRY(check_step("kda_lattn_step", dims->B, dims->T, dims->N, dims->cu_seqlens_dev, dims->cu_seqlens_host, slots, S));
  REQUIRE(q, "q");
  REQUIRE(k, "k");
  REQUIRE(v, "v");
  REQUIRE(g, "g");
  REQUIRE(state, "state");
  REQUIRE(o, "o");
  kda::LinStepArgs a{};
  a.B = dims->B;
  a.H = dims->H;
  a.HV = dims->HV;
  a.K = dims->K;
  a.V = dims->V;
  a.slots_n = S;
  a.g_const = dims->g_const;
  a.scale = dims->scale;
  a.q_row = p.q_row;
  a.k_row = p.k_row;
  a.v_row = p.v_row;
  a.q = q;
  a.k = k;
  a.v = v;
  a.g = g;
  a.slots = slots;
  a.state = state;
  a.o = o;
  return hip_status(kda::launch_lin_step(dims->dtype, a, static_cast<hipStream_t>(stream)), "kda_lattn_step");
}

// ---- window attention

namespace {

kda_status win_check(const kda_wattn_dims* d, bool launching, Tokens* t, kda::WinArgs* a) {
  if (d == nullptr) return fail(KDA_EINVAL, "dims is NULL");
  TRY(check_tokens(d->B, d->T, d->N, d->cu_seqlens_dev, d->cu_seqlens_host, launching, t));
  if (d->H <= 0 || d->HK <= 0 || d->D <= 0) return fail(KDA_EINVAL, "dims must be positive (H=%d HK=%d D=%d)", d->H, d->HK, d->D);
  if (d->H % d->HK != 0) return fail(KDA_EINVAL, "H (%d) must be a multiple of HK (%d)", d->H, d->HK);
  if (d->D > 256) return fail(KDA_EUNSUPPORTED, "D must be at most 256, got %d", d->D);
  if (d->H > 1 << 16) return fail(KDA_EINVAL, "too many heads (%d)", d->H);
  if (d->window < 1 || d->window > 1 << 30) return fail(KDA_EINVAL, "window must be in 1 .. 2^30, got %d", d->window);
  if (d->sinks < 0 || d->sinks > 1024) return fail(KDA_EINVAL, "sinks must be in 0 .. 1024, got %d", d->sinks);
  if (!std::isfinite(d->scale)) return fail(KDA_EINVAL, "scale must be finite");
  TRY(check_dtype(d->dtype));
  *a = kda::WinArgs{};
  TRY(tile_row(d->q_row, (int64_t)d->H * d->D, "q", &a->q_row));
  TRY(tile_row(d->k_row, (int64_t)d->HK * d->D, "k", &a->k_row));
  TRY(tile_row(d->v_row, (int64_t)d->HK * d->D, "v", &a->v_row));
  a->sq = t->sq;
  a->H = d->H;
  a->HK = d->HK;
  a->D = d->D;
  a->window = d->window;
  a->sinks = d->sinks;
  a->scale = d->scale;
  return KDA_OK;
}

// The grids over whole sequences: runs of 64 tokens at the least.
kda_status win_grids(const kda_wattn_dims* d, const Tokens& t) {
  if ((t.sq.total / 64 + d->N) * d->H > kMaxBlocks) return fail(KDA_EINVAL, "too many tokens (%lld of %d heads)", (long long)t.sq.total, d->H);
  return KDA_OK;
}

void win_vec(kda::WinArgs* a, int dtype) {
  const int ev = dtype == KDA_F32 ? 4 : 8;
  a->vec = a->D % ev == 0 && a->q_row % ev == 0 && a->k_row % ev == 0 && a->v_row % ev == 0 &&
           aligned({a->q, a->k, a->v, a->o, a->out, a->dout, a->dq, a->dk, a->dv}, 16);
}

struct WinLayout {
  size_t delta = 0, part = 0, total = 0;
  int64_t parts = 0;
  int part_len = 0;
};

WinLayout win_layout(const kda_wattn_dims* d, const Tokens& t) {
  WinLayout l;
  size_t o = 0;
  l.delta = o;
  o = align_up(o + (size_t)t.sq.total * d->H * sizeof(float));
  if (d->sinks > 0 && t.longest > d->window) {
    // queries of a part behind the window: two workgroups for each CU, at least two blocks for each wave, and at most 64 parts
    // to be joined where sequences are long
    const int64_t tiles = (int64_t)((d->sinks + 15) / 16) * d->HK;
    const int64_t least = std::min<int64_t>(256, std::max<int64_t>(64, t.sq.total * tiles / 512 / 32 * 32));
    l.part_len = (int)std::max<int64_t>(least, ((t.longest - d->window + 63) / 64 + 31) / 32 * 32);
    l.parts = count_runs(d->cu_seqlens_host, d->N, d->T, l.part_len, d->window);
    l.part = o;
    o = align_up(o + (size_t)(l.parts + d->N) * d->sinks * d->HK * 2 * d->D * sizeof(float));
  }
  l.total = o;
  return l;
}

// The backward's: also those of the first tokens where sequences are longer than the window.
kda_status win_bwd_grids(const kda_wattn_dims* d, const Tokens& t, const WinLayout& l) {
  TRY(win_grids(d, t));
  if (l.parts > 0 && ((int64_t)d->N * d->sinks * d->HK > kMaxBlocks || l.parts * ((d->sinks + 15) / 16) * d->HK > kMaxBlocks))
    return fail(KDA_EINVAL, "too many first tokens (%d of %d sequences and %d key heads)", d->sinks, d->N, d->HK);
  return KDA_OK;
}

struct StepPlan {
  int rows, splits;
  size_t bytes;
};
kda_status win_step_check(const kda_wattn_dims* d, kda::WinArgs* c, StepPlan* p) {
  Tokens t;
  TRY(win_check(d, false, &t, c));
  if (d->B > kMaxStepRows || d->T != 1 || d->N != d->B || d->cu_seqlens_dev != nullptr || d->cu_seqlens_host != nullptr)
    return fail(KDA_EINVAL, "kda_wattn_step takes one token per sequence (T = 1, N = B <= %d, no cu_seqlens)", kMaxStepRows);
  const int total = d->sinks + d->window;
  p->rows = kda::win_step_rows(d->B, d->HK, total);
  p->splits = (total + p->rows - 1) / p->rows;
  // the step's workgroups (a row of sequences each) and, where a key head's rows are dealt to several, the join's
  if ((int64_t)p->splits * d->H > kMaxBlocks || (p->splits > 1 && (int64_t)d->B * d->H > kMaxBlocks))
    return fail(KDA_EINVAL, "too many heads (%d of %d sequences)", d->H, d->B);
  p->bytes = p->splits > 1 ? align_up((size_t)d->B * d->H * p->splits * (d->D + 2) * sizeof(float)) : 0;
  return KDA_OK;
}

}  // namespace

KDA_EXPORT kda_status kda_wattn_fwd(const kda_wattn_dims* dims, const void* q, const void* k, const void* v, void* o,
                                    float* lse, void* k_cache, void* v_cache, void* stream) {
  Tokens t;
  kda::WinArgs a;
  TRY(win_check(dims, true, &t, &a));
  TRY(win_grids(dims, t));
  if (t.sq.total > 0) {
    REQUIRE(q, "q");
    REQUIRE(k, "k");
    REQUIRE(v, "v");
    REQUIRE(o, "o");
  }
  if ((k_cache == nullptr) != (v_cache == nullptr)) return fail(KDA_EINVAL, "k_cache and v_cache must be both given or both NULL");
  if (k_cache != nullptr && (int64_t)dims->N * ((int64_t)dims->sinks + dims->window) > kMaxBlocks)
    return fail(KDA_EINVAL, "too many cache rows (%d of %lld)", dims->N, (long long)dims->sinks + dims->window);
  a.q = q;
  a.k = k;
  a.v = v;
  a.o = o;
  a.lse = lse;
  win_vec(&a, dims->dtype);
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (t.sq.total > 0) {
    const kda::WinPlan p = kda::win_plan(dims->dtype, a.D, t.sq.total, dims->N, a.H, a.HK);
    a.blocks = count_runs(dims->cu_seqlens_host, dims->N, dims->T, p.qrows, 0);
    TRY(hip_status(kda::launch_win_fwd(dims->dtype, a, p.qrows, st), "kda_wattn_fwd"));
  }
  if (k_cache != nullptr) TRY(hip_status(kda::launch_win_cache(dims->dtype, a, k_cache, v_cache, st), "kda_wattn_fwd"));
  return KDA_OK;
}

KDA_EXPORT size_t kda_wattn_bwd_workspace_bytes(const kda_wattn_dims* dims) {
  Tokens t;
  kda::WinArgs a;
  if (win_check(dims, false, &t, &a) != KDA_OK) return 0;
  const WinLayout l = win_layout(dims, t);
  return win_bwd_grids(dims, t, l) == KDA_OK ? l.total : 0;
}

KDA_EXPORT kda_status kda_wattn_bwd(const kda_wattn_dims* dims, const void* q, const void* k, const void* v,
                                    const void* o, const float* lse, const void* dout, void* dq, void* dk, void* dv,
                                    void* workspace, size_t ws_bytes, void* stream) {
  Tokens t;
  kda::WinArgs a;
  TRY(win_check(dims, true, &t, &a));
  const WinLayout l = win_layout(dims, t);
  TRY(win_bwd_grids(dims, t, l));
  if (t.sq.total == 0) return KDA_OK;
  REQUIRE(q, "q");
  REQUIRE(k, "k");
  REQUIRE(v, "v");
  REQUIRE(o, "o");
  REQUIRE(lse, "lse");
  REQUIRE(dout, "do");
  REQUIRE(dq, "dq");
  REQUIRE(dk, "dk");
  REQUIRE(dv, "dv");
  TRY(check_ws(workspace, ws_bytes, l.total));
  char* ws = static_cast<char*>(workspace);
  a.q = q;
  a.k = k;
  a.v = v;
  a.out = o;
  a.dout = dout;
  a.lse_in = lse;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  a.delta = reinterpret_cast<float*>(ws + l.delta);
  a.part = reinterpret_cast<float*>(ws + l.part);
  a.part_len = l.part_len;
  a.parts = l.parts;
  win_vec(&a, dims->dtype);
  hipStream_t st = static_cast<hipStream_t>(stream);
  const kda::WinPlan p = kda::win_plan(dims->dtype, a.D, t.sq.total, dims->N, a.H, a.HK);
  a.blocks = count_runs(dims->cu_seqlens_host, dims->N, dims->T, p.qrows, 0);
  TRY(hip_status(kda::launch_win_dq(dims->dtype, a, p.qrows, st), "kda_wattn_bwd"));
  a.blocks = count_runs(dims->cu_seqlens_host, dims->N, dims->T, p.krows, 0);
  TRY(hip_status(kda::launch_win_dkv(dims->dtype, a, p.krows, st), "kda_wattn_bwd"));
  if (l.parts > 0) TRY(hip_status(kda::launch_win_sinks(dims->dtype, a, st), "kda_wattn_bwd"));
  return KDA_OK;
}

KDA_EXPORT size_t kda_wattn_step_workspace_bytes(const kda_wattn_dims* dims) {
  kda::WinArgs c;
  StepPlan p;
  if (win_step_check(dims, &c, &p) != KDA_OK) return (size_t)-1;
  return p.bytes;
}

KDA_EXPORT kda_status kda_wattn_step(const kda_wattn_dims* dims, const void* q, const void* k, const void* v,
                                     const int32_t* pos, const int32_t* slots, int32_t S, void* k_cache, void* v_cache,
                                     void* o, void* workspace, size_t ws_bytes, void* stream) {
  kda::WinArgs c;
  StepPlan p;
  TRY(win_step_check(dims, &c, &p));
  TRY(check_step("kda_wattn_step", dims->B, dims->T, dims->N, dims->cu_seqlens_dev, dims->cu_seqlens_host, slots, S));
  REQUIRE(q, "q");
  REQUIRE(k, "k");
  REQUIRE(v, "v");
  REQUIRE(pos, "pos");
  REQUIRE(k_cache, "k_cache");
  REQUIRE(v_cache, "v_cache");
  REQUIRE(o, "o");
  TRY(check_ws(workspace, ws_bytes, p.bytes));
  kda::WinStepArgs a{};
  a.B = dims->B;
  a.H = dims->H;
  a.HK = dims->HK;
  a.D = dims->D;
  a.window = dims->window;
  a.sinks = dims->sinks;
  a.slots_n = S;
  a.scale = dims->scale;
  a.q_row = c.q_row;
  a.k_row = c.k_row;
  a.v_row = c.v_row;
  a.q = q;
  a.k = k;
  a.v = v;
  a.pos = pos;
  a.slots = slots;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.o = o;
  const int ev = dims->dtype == KDA_F32 ? 4 : 8;
  a.vec = a.D % ev == 0 && a.q_row % ev == 0 && aligned({q, k_cache, v_cache}, 16);
  a.rows = p.rows;
  a.splits = p.splits;
  a.part = static_cast<float*>(workspace);
  return hip_status(kda::launch_win_step(dims->dtype, a, static_cast<hipStream_t>(stream)), "kda_wattn_step");
}
