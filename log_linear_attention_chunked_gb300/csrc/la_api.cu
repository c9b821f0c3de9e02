// C ABI entry points of linear attention with a decay per head and of rotary
// positions: argument checks, launch.
#include <cmath>

#include "la.cuh"

using namespace llattn;

static ll_status check_la_shape(const ll_la_shape* s) {
  if (!s) return LL_ERR_INVALID_ARG;
  if (s->B < 1 || s->H < 1 || s->Hk < 1 || s->T < 1 || s->n_seqs < 0) return LL_ERR_INVALID_ARG;
  if (s->H % s->Hk != 0 || (s->n_seqs > 0 && s->B != 1)) return LL_ERR_INVALID_ARG;
  if (s->io != LL_F32 && s->io != LL_BF16) return LL_ERR_INVALID_ARG;
  if (s->per_head != 0 && s->per_head != 1) return LL_ERR_INVALID_ARG;
  if (!std::isfinite(s->scale)) return LL_ERR_INVALID_ARG;
  if (!head_dim_ok(s->dk) || !head_dim_ok(s->dv)) return LL_ERR_UNSUPPORTED;
  // tokens are counted in 31 bits, in whole segments and a few tiles ahead
  if (s->T > 0x7fffffff - 1024) return LL_ERR_UNSUPPORTED;
  // CTAs are counted in 31 bits: at most (sequences or 16-token pieces) x heads x 8 of them
  const long long units = s->n_seqs ? (long long)s->T / 16 + s->n_seqs : (long long)s->B * ((s->T + 15ll) / 16);
  if (units >= (1ll << 31) || units * s->H >= (1ll << 26)) return LL_ERR_UNSUPPORTED;
  return LL_OK;
}

static LaArgs la_args(const ll_la_shape* s) {
  LaArgs a{};
  a.B = s->B;
  a.H = s->H;
  a.Hk = s->Hk;
  a.T = s->T;
  a.dk = s->dk;
  a.dv = s->dv;
  a.n_seqs = s->n_seqs;
  a.io = s->io;
  a.per_head = s->per_head;
  a.scale = s->scale;
  return a;
}

static ll_status check_workspace(size_t need, const void* ws, size_t bytes) {
  if (need == 0) return LL_OK;
  if (!ws || bytes < need || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return LL_ERR_WORKSPACE;
  return LL_OK;
}

extern "C" {

size_t ll_la_fwd_workspace_size(const ll_la_shape* s) {
  return check_la_shape(s) == LL_OK ? la_fwd_workspace(la_args(s)) : 0;
}

int ll_la_fwd_launches(const ll_la_shape* s) { return check_la_shape(s) == LL_OK ? la_fwd_launches(la_args(s)) : 0; }

ll_status ll_la_fwd(const ll_la_shape* s, const int32_t* seq_starts, const void* q, const void* k, const void* v,
                    const float* log_alpha, const float* state_in, void* o, float* state_out, void* workspace,
                    size_t ws_bytes, void* stream) {
  const ll_status st = check_la_shape(s);
  if (st != LL_OK) return st;
  if ((seq_starts != nullptr) != (s->n_seqs > 0)) return LL_ERR_INVALID_ARG;
  const size_t es = s->io == LL_F32 ? 4 : 2, rows = (size_t)s->B * s->H * s->T, krows = (size_t)s->B * s->Hk * s->T;
  const size_t states = (size_t)(s->n_seqs ? s->n_seqs : s->B) * s->H * s->dv * s->dk * 4;
  const Range in[6] = {{q, krows * s->dk * es}, {k, krows * s->dk * es}, {v, rows * s->dv * es},
                       {log_alpha, s->per_head ? (size_t)s->H * 4 : rows * 4}, {state_in, states},
                       {seq_starts, (size_t)(s->n_seqs + 1) * 4}};
  const Range out[2] = {{o, rows * s->dv * es}, {state_out, states}};
  for (int i = 0; i < 6; ++i)
    if ((i < 4 && !in[i].p) || !aligned16(in[i].p)) return LL_ERR_INVALID_ARG;
  if (!o || !aligned16(o) || !aligned16(state_out)) return LL_ERR_INVALID_ARG;
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 6; ++j)
      if (ranges_overlap(out[i], in[j]) && !(i == 1 && j == 4 && state_in == state_out)) return LL_ERR_INVALID_ARG;
  if (ranges_overlap(out[0], out[1])) return LL_ERR_INVALID_ARG;
  LaArgs a = la_args(s);
  const ll_status wst = check_workspace(la_fwd_workspace(a), workspace, ws_bytes);
  if (wst != LL_OK) return wst;
  a.seq_starts = seq_starts;
  a.q = q;
  a.k = k;
  a.v = v;
  a.log_alpha = log_alpha;
  a.state_in = state_in;
  a.o = o;
  a.state_out = state_out;
  a.ws = workspace;
  a.ws_bytes = ws_bytes;
  a.stream = static_cast<cudaStream_t>(stream);
  a.err = err_word();
  if (!a.err) return LL_ERR_CUDA;
  return la_fwd_launch(a);
}

size_t ll_la_bwd_workspace_size(const ll_la_shape* s) {
  return check_la_shape(s) == LL_OK ? la_bwd_workspace(la_args(s)) : 0;
}

int ll_la_bwd_launches(const ll_la_shape* s) { return check_la_shape(s) == LL_OK ? la_bwd_launches(la_args(s)) : 0; }

ll_status ll_la_bwd(const ll_la_shape* s, const int32_t* seq_starts, const void* q, const void* k, const void* v,
                    const float* log_alpha, const float* state_in, const void* dout, const float* dstate_out, void* dq,
                    void* dk, void* dv, float* dlog_alpha, float* dstate_in, void* workspace, size_t ws_bytes,
                    void* stream) {
  const ll_status st = check_la_shape(s);
  if (st != LL_OK) return st;
  if ((seq_starts != nullptr) != (s->n_seqs > 0)) return LL_ERR_INVALID_ARG;
  const size_t es = s->io == LL_F32 ? 4 : 2, rows = (size_t)s->B * s->H * s->T, krows = (size_t)s->B * s->Hk * s->T;
  const size_t states = (size_t)(s->n_seqs ? s->n_seqs : s->B) * s->H * s->dv * s->dk * 4;
  const size_t gates = s->per_head ? (size_t)s->H * 4 : rows * 4;
  const Range in[8] = {{q, krows * s->dk * es}, {k, krows * s->dk * es}, {v, rows * s->dv * es},
                       {log_alpha, gates},      {dout, rows * s->dv * es}, {state_in, states},
                       {dstate_out, states},    {seq_starts, (size_t)(s->n_seqs + 1) * 4}};
  const Range out[5] = {{dq, krows * s->dk * es}, {dk, krows * s->dk * es}, {dv, rows * s->dv * es},
                        {dlog_alpha, gates},      {dstate_in, states}};
  for (int i = 0; i < 8; ++i)
    if ((i < 5 && !in[i].p) || !aligned16(in[i].p)) return LL_ERR_INVALID_ARG;
  for (int i = 0; i < 5; ++i) {
    if ((i < 4 && !out[i].p) || !aligned16(out[i].p)) return LL_ERR_INVALID_ARG;
    for (int j = 0; j < 8; ++j)
      if (ranges_overlap(out[i], in[j]) && !(i == 4 && j == 6 && dstate_in == dstate_out)) return LL_ERR_INVALID_ARG;
    for (int j = i + 1; j < 5; ++j)
      if (ranges_overlap(out[i], out[j])) return LL_ERR_INVALID_ARG;
  }
  LaArgs a = la_args(s);
  const ll_status wst = check_workspace(la_bwd_workspace(a), workspace, ws_bytes);
  if (wst != LL_OK) return wst;
  a.seq_starts = seq_starts;
  a.q = q;
  a.k = k;
  a.v = v;
  a.log_alpha = log_alpha;
  a.state_in = state_in;
  a.dout = dout;
  a.dstate_out = dstate_out;
  a.dq = dq;
  a.dkey = dk;
  a.dval = dv;
  a.dlog_alpha = dlog_alpha;
  a.dstate_in = dstate_in;
  a.ws = workspace;
  a.ws_bytes = ws_bytes;
  a.stream = static_cast<cudaStream_t>(stream);
  a.err = err_word();
  if (!a.err) return LL_ERR_CUDA;
  return la_bwd_launch(a);
}

static ll_status check_rope(const ll_rope* r, int d) {
  if (r->rot < 2 || r->rot > d || r->rot % 2 != 0) return LL_ERR_INVALID_ARG;
  if (r->interleaved != 0 && r->interleaved != 1) return LL_ERR_INVALID_ARG;
  if (!std::isfinite(r->amp) || !r->inv_freq || !aligned16(r->inv_freq)) return LL_ERR_INVALID_ARG;
  return LL_OK;
}

ll_status ll_la_decode_step(int B, int H, int Hk, int dk, int dv, ll_dtype io, int per_head, float scale,
                            const int64_t* slots, int n_slots, const ll_rope* rope, const int64_t* positions,
                            const void* q, const void* k, const void* v, const float* log_alpha, float* states, void* o,
                            void* stream) {
  if (B < 1 || H < 1 || Hk < 1 || H % Hk != 0 || n_slots < 1) return LL_ERR_INVALID_ARG;
  if (!slots && n_slots < B) return LL_ERR_INVALID_ARG;
  if (io != LL_F32 && io != LL_BF16) return LL_ERR_INVALID_ARG;
  if (per_head != 0 && per_head != 1) return LL_ERR_INVALID_ARG;
  if (!std::isfinite(scale)) return LL_ERR_INVALID_ARG;
  if (!head_dim_ok(dk) || !head_dim_ok(dv)) return LL_ERR_UNSUPPORTED;
  if ((long long)B * H >= (1ll << 26)) return LL_ERR_UNSUPPORTED;
  if (!q || !k || !v || !log_alpha || !states || !o) return LL_ERR_INVALID_ARG;
  if ((rope != nullptr) != (positions != nullptr)) return LL_ERR_INVALID_ARG;
  if (rope) {
    const ll_status st = check_rope(rope, dk);
    if (st != LL_OK) return st;
  }
  if (!aligned16(slots) || !aligned16(positions) || !aligned16(q) || !aligned16(k) || !aligned16(v) ||
      !aligned16(log_alpha) || !aligned16(states) || !aligned16(o))
    return LL_ERR_INVALID_ARG;
  const size_t es = io == LL_F32 ? 4 : 2;
  const size_t bk = (size_t)B * Hk * dk * es, bv = (size_t)B * H * dv * es;
  const Range in[7] = {{q, bk}, {k, bk}, {v, bv}, {log_alpha, (size_t)(per_head ? 1 : B) * H * 4}, {slots, (size_t)B * 8},
                       {positions, (size_t)B * 8}, {rope ? rope->inv_freq : nullptr, rope ? (size_t)rope->rot * 2 : 0}};
  const Range out[2] = {{o, bv}, {states, (size_t)n_slots * H * dv * dk * 4}};
  for (const Range& w : out)
    for (const Range& r : in)
      if (ranges_overlap(w, r)) return LL_ERR_INVALID_ARG;
  if (ranges_overlap(out[0], out[1])) return LL_ERR_INVALID_ARG;
  unsigned* ew = err_word();
  if (!ew) return LL_ERR_CUDA;
  LaStepArgs a{};
  a.B = B;
  a.H = H;
  a.Hk = Hk;
  a.dk = dk;
  a.dv = dv;
  a.io = io;
  a.per_head = per_head;
  a.scale = scale;
  a.slots = slots;
  a.n_slots = n_slots;
  a.q = q;
  a.k = k;
  a.v = v;
  a.log_alpha = log_alpha;
  a.states = states;
  if (rope) a.rope = LaRope{rope->rot, rope->interleaved, rope->inv_freq, rope->amp};
  a.positions = positions;
  a.o = o;
  a.stream = static_cast<cudaStream_t>(stream);
  a.err = ew;
  return la_step_launch(a);
}

static ll_status rope_call(bool back, int B, int H, int Hk, int T, int d, ll_dtype io, const ll_rope* rope,
                           const int64_t* positions, const void* q, const void* k, void* q_out, void* k_out,
                           void* stream) {
  if (!rope || B < 1 || H < 1 || T < 1 || !q || !q_out) return LL_ERR_INVALID_ARG;
  if ((k != nullptr) != (k_out != nullptr) || (k ? Hk < 1 : Hk != 0)) return LL_ERR_INVALID_ARG;
  if (io != LL_F32 && io != LL_BF16) return LL_ERR_INVALID_ARG;
  if (!head_dim_ok(d)) return LL_ERR_UNSUPPORTED;
  const ll_status st = check_rope(rope, d);
  if (st != LL_OK) return st;
  if ((long long)H + Hk > 0xffff || T > 0x7fffffff - 1024 || (long long)B * T >= (1ll << 31)) return LL_ERR_UNSUPPORTED;
  if (!aligned16(positions) || !aligned16(q) || !aligned16(k) || !aligned16(q_out) || !aligned16(k_out))
    return LL_ERR_INVALID_ARG;
  const size_t row = (size_t)B * T * d * (io == LL_F32 ? 4 : 2);
  const Range in[4] = {{q, row * H}, {k, row * Hk}, {positions, (size_t)B * T * 8}, {rope->inv_freq, (size_t)rope->rot * 2}};
  const Range out[2] = {{q_out, row * H}, {k_out, row * Hk}};
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 4; ++j)
      if (ranges_overlap(out[i], in[j]) && !(i == j && out[i].p == in[j].p)) return LL_ERR_INVALID_ARG;
  if (ranges_overlap(out[0], out[1])) return LL_ERR_INVALID_ARG;
  RopeArgs a{B, H, Hk, T, d, io, LaRope{rope->rot, rope->interleaved, rope->inv_freq, rope->amp}, positions, q, k, q_out,
             k_out, back, static_cast<cudaStream_t>(stream)};
  return rope_launch(a);
}

ll_status ll_rope_fwd(int B, int H, int Hk, int T, int d, ll_dtype io, const ll_rope* rope, const int64_t* positions,
                      const void* q, const void* k, void* q_out, void* k_out, void* stream) {
  return rope_call(false, B, H, Hk, T, d, io, rope, positions, q, k, q_out, k_out, stream);
}

ll_status ll_rope_bwd(int B, int H, int Hk, int T, int d, ll_dtype io, const ll_rope* rope, const int64_t* positions,
                      const void* dq_out, const void* dk_out, void* dq, void* dk, void* stream) {
  return rope_call(true, B, H, Hk, T, d, io, rope, positions, dq_out, dk_out, dq, dk, stream);
}

ll_status ll_rope_freqs(int rot, double base, double factor, double length, double slow_turns, double fast_turns,
                        float* inv_freq) {
  if (rot < 2 || rot % 2 != 0 || rot > 128 || !inv_freq) return LL_ERR_INVALID_ARG;
  if (!(base > 1.) || !std::isfinite(base) || !(factor >= 1.) || !std::isfinite(factor)) return LL_ERR_INVALID_ARG;
  const bool ramp = length != 0.;
  if (ramp && (!(length > 0.) || !std::isfinite(length) || !(slow_turns >= 0.) || !(fast_turns > slow_turns) ||
               !std::isfinite(fast_turns)))
    return LL_ERR_INVALID_ARG;
  const double turn = 6.283185307179586476925;
  for (int i = 0; i < rot / 2; ++i) {
    const double f = std::pow(base, -2. * i / rot);
    double keep = 0.;
    if (ramp) keep = std::fmin(1., std::fmax(0., (length * f / turn - slow_turns) / (fast_turns - slow_turns)));
    inv_freq[i] = (float)(f * keep + f / factor * (1. - keep));
  }
  return LL_OK;
}

}  // extern "C"
