// attn_api.cu -- host side of packed causal attention: argument checks,
// tensor maps, scratch and the launch sequence.
#include <cmath>

#include "attn.h"
#include "host_util.h"

namespace flce {
namespace {

// A [T, heads, D] operand: address and strides, with the stride of an axis of
// one element (which may be anything) replaced by a valid one.
struct Operand {
  const void* p;
  int64_t token, head;
};

int operand(Operand* out, const char* name, const void* p, int64_t token, int64_t head, int64_t T,
            int heads, int D) {
  if (!p) return host_error(FLCE_ERR_ARG, "%s is null", name);
  if (heads == 1) head = D;
  if (T == 1) token = head * heads;
  if (token <= 0 || head <= 0)
    return host_error(FLCE_ERR_ARG, "%s: strides must be positive", name);
  if (token % 8 != 0 || head % 8 != 0 || !aligned16(p))
    return host_error(FLCE_ERR_ALIGN,
                      "%s must be 16-byte aligned with strides that are multiples of 8", name);
  if (token >= (int64_t{1} << 38) || head >= (int64_t{1} << 38))
    return host_error(FLCE_ERR_ARG, "%s: stride too large", name);
  *out = Operand{p, token, head};
  return FLCE_OK;
}

// Whether operands of `na` and `nb` heads share an element, as far as can be told: by
// their address ranges, first elements and, for equal token strides, every pair of
// heads (interleaved slices of one buffer share none).
bool shared(const Operand& a, int na, const Operand& b, int nb, int64_t T, int D) {
  using wide = __int128;  // strides below 2^38, T below 2^31
  const wide a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  const wide row = 2 * D, s = 2 * wide{a.token};
  const wide wa = 2 * wide{na - 1} * a.head + row, wb = 2 * wide{nb - 1} * b.head + row;
  if (a0 + (T - 1) * s + wa <= b0 || b0 + 2 * (T - 1) * wide{b.token} + wb <= a0) return false;
  if (a0 == b0) return true;
  if (a.token != b.token || wide{na} * nb > (1 << 16)) return false;  // not told
  auto mod = [&](wide x) { return (x % s + s) % s; };
  const wide off = mod(b0 - a0);
  if (off >= wa && off + wb <= s) return false;  // beside each other in every token
  for (int i = 0; i < na; ++i)
    for (int j = 0; j < nb; ++j) {
      const wide d = b0 + 2 * wide{j} * b.head - (a0 + 2 * wide{i} * a.head);
      const wide r = mod(d), t = (d - r) / s;  // t tokens and r bytes apart
      if ((r < row && t < T && -t < T) || (s - r < row && t + 1 < T && -t - 1 < T)) return true;
    }
  return false;
}

int tensor_map(CUtensorMap* m, const Operand& t, int64_t T, int heads, int D, const char* name) {
  const uint64_t dims[3] = {static_cast<uint64_t>(D), static_cast<uint64_t>(heads),
                            static_cast<uint64_t>(T)};
  const uint64_t pitch[2] = {static_cast<uint64_t>(t.head) * 2, static_cast<uint64_t>(t.token) * 2};
  const uint32_t box[3] = {64, 1, kTile};
  return host_tensor_map(m, t.p, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, dims, pitch, box, name);
}

int attention(const flce_attn* a, const flce_opts* opts, bool backward) {
  host_clear_error();
  const flce_opts o = opts_or_default(opts);
  if (!a) return host_error(FLCE_ERR_ARG, "null flce_attn");
  if (o.dtype != FLCE_BF16)
    return host_error(FLCE_ERR_ARG, "attention takes bf16 inputs (dtype %d)", o.dtype);
  if (a->T < 0 || a->T >= (int64_t{1} << 31) - 256 || a->batch < 0 ||
      a->batch >= (int64_t{1} << 30))
    return host_error(FLCE_ERR_ARG, "sizes must satisfy 0 <= T < 2^31 - 256, 0 <= batch < 2^30");
  if (a->heads_kv < 1 || a->heads_q < 1 || a->heads_q % a->heads_kv != 0)
    return host_error(FLCE_ERR_ARG, "heads_kv must be positive and divide heads_q");
  const int D = a->head_dim;
  if (D < 8 || D > 128 || D % 8 != 0)
    return host_error(FLCE_ERR_ARG, "head_dim must be a multiple of 8 in 8 .. 128 (got %d)", D);
  if (!(a->scale > 0.f) || std::isinf(a->scale))
    return host_error(FLCE_ERR_ARG, "scale must be positive and finite");
  if (!a->cu_seqlens) return host_error(FLCE_ERR_ARG, "cu_seqlens is null");
  const int64_t T = a->T;
  const int unit = backward ? 1 : 2;
  const int64_t max_tiles = T / (kTile * unit) + a->batch;
  if ((T / kTile + a->batch) * a->heads_q >= (int64_t{1} << 31))
    return host_error(FLCE_ERR_ARG, "(T / 128 + batch) * heads_q must be below 2^31");
  int rc = FLCE_OK;
  Operand q{}, k{}, v{}, oo{}, dO{}, dq{}, dk{}, dv{};
  if (T > 0) {
    if ((rc = operand(&q, "q", a->q, a->q_token, a->q_head, T, a->heads_q, D))) return rc;
    if ((rc = operand(&k, "k", a->k, a->k_token, a->k_head, T, a->heads_kv, D))) return rc;
    if ((rc = operand(&v, "v", a->v, a->v_token, a->v_head, T, a->heads_kv, D))) return rc;
    if ((rc = operand(&oo, "o", a->o, a->o_token, a->o_head, T, a->heads_q, D))) return rc;
    if (!a->lse) return host_error(FLCE_ERR_ARG, "lse is null");
    if (backward) {
      if ((rc = operand(&dO, "dO", a->dO, a->dO_token, a->dO_head, T, a->heads_q, D))) return rc;
      if ((rc = operand(&dq, "dq", a->dq, a->dq_token, a->dq_head, T, a->heads_q, D))) return rc;
      if ((rc = operand(&dk, "dk", a->dk, a->dk_token, a->dk_head, T, a->heads_kv, D))) return rc;
      if ((rc = operand(&dv, "dv", a->dv, a->dv_token, a->dv_head, T, a->heads_kv, D))) return rc;
    }
    // An output over what other CTAs, or the same one, still read; o over q too (a
    // second pass over a unit, see attn_fwd.cu).  The gradients may take o's place:
    // only delta is formed from it, before the first of them is written.
    const struct { const char* name; Operand t; int heads; } in[] = {
        {"q", q, a->heads_q}, {"k", k, a->heads_kv}, {"v", v, a->heads_kv}, {"dO", dO, a->heads_q}},
        out[] = {{"dq", dq, a->heads_q}, {"dk", dk, a->heads_kv}, {"dv", dv, a->heads_kv}};
    auto apart = [&](const auto& x, const auto& y) {
      return shared(x.t, x.heads, y.t, y.heads, T, D)
                 ? host_error(FLCE_ERR_ARG, "%s overlaps %s", x.name, y.name)
                 : FLCE_OK;
    };
    if (backward) {
      for (int i = 0; i < 3; ++i) {
        for (const auto& x : in)
          if ((rc = apart(out[i], x))) return rc;
        for (int j = 0; j < i; ++j)
          if ((rc = apart(out[i], out[j]))) return rc;
      }
    } else {
      for (int j = 0; j < 3; ++j)
        if (shared(oo, a->heads_q, in[j].t, in[j].heads, T, D))
          return host_error(FLCE_ERR_ARG, "o overlaps %s", in[j].name);
    }
  }
  int sms = 0;
  if ((rc = host_device(&sms))) return rc;
  CUtensorMap mq, mk, mv, mO;
  if (T > 0) {
    if ((rc = tensor_map(&mq, q, T, a->heads_q, D, "q"))) return rc;
    if ((rc = tensor_map(&mk, k, T, a->heads_kv, D, "k"))) return rc;
    if ((rc = tensor_map(&mv, v, T, a->heads_kv, D, "v"))) return rc;
    if (backward && (rc = tensor_map(&mO, dO, T, a->heads_q, D, "dO"))) return rc;
  }
  AttnParams p{};
  p.cu = a->cu_seqlens;
  p.B = static_cast<int32_t>(a->batch);
  p.T = static_cast<int32_t>(T);
  p.Hq = a->heads_q;
  p.Hkv = a->heads_kv;
  p.D = D;
  p.scale = a->scale;
  p.max_tiles = static_cast<int32_t>(max_tiles);
  p.unit = unit;
  p.max_depth = static_cast<int32_t>((T + kTile * unit - 1) / (kTile * unit));
  const size_t b_tiles = T > 0 ? round256(static_cast<size_t>(max_tiles) * sizeof(AttnTile)) : 0;
  const size_t b_bucket = round256((static_cast<size_t>(p.max_depth) + 2) * 4);
  const size_t b_delta =
      backward ? round256(static_cast<size_t>(a->heads_q) * static_cast<size_t>(T) * 4) : 0;
  const bool direct = !backward && a->batch >= 1 && a->batch <= kDirectSeqs &&
                      max_tiles * a->heads_q <= sms;
  // without tokens the plan only checks the offsets, for a caller who looks at the status
  const bool planned = T > 0 ? !direct : o.sync || o.status_dev;
  StepCall call;
  if ((rc = call.begin(o, planned ? 256 + b_tiles + b_bucket + b_delta : 0,
                       planned ? StepCall::kKernelClears : StepCall::kIfAsked)))
    return rc;
  if (planned) {
    uint8_t* w = call.scratch;
    p.n_tiles = reinterpret_cast<int32_t*>(w);
    p.tiles = reinterpret_cast<AttnTile*>(w + 256);
    p.bucket = reinterpret_cast<int32_t*>(w + 256 + b_tiles);
    p.delta = backward ? reinterpret_cast<float*>(w + 256 + b_tiles + b_bucket) : nullptr;
  }
  p.lse = a->lse;
  p.status = call.status;
  p.k = AttnOut{const_cast<void*>(a->k), k.token, k.head};
  p.v = AttnOut{const_cast<void*>(a->v), v.token, v.head};
  p.o = AttnOut{a->o, oo.token, oo.head};
  p.dO = AttnOut{const_cast<void*>(a->dO), dO.token, dO.head};
  p.dq = AttnOut{a->dq, dq.token, dq.head};
  p.dk = AttnOut{a->dk, dk.token, dk.head};
  p.dv = AttnOut{a->dv, dv.token, dv.head};
  cudaError_t e = planned ? launch_attn_plan(p, backward, sms, call.stream) : cudaSuccess;
  if (T > 0 && max_tiles > 0) {
    if (backward) {
      if (e == cudaSuccess) e = launch_attn_dkdv(mq, mk, mv, mO, p, sms, call.stream);
      if (e == cudaSuccess) e = launch_attn_dq(mq, mk, mv, mO, p, call.stream);
    } else if (e == cudaSuccess) {
      e = launch_attn_fwd(mq, mk, mv, p, sms, call.stream);
    }
  }
  if (e != cudaSuccess) rc = host_cuda_error(e, backward ? "flce_attn_bwd" : "flce_attn_fwd");
  return call.end(rc);
}

}  // namespace
}  // namespace flce

extern "C" {

int flce_attn_fwd(const flce_attn* a, const flce_opts* opts) {
  return flce::attention(a, opts, false);
}

int flce_attn_bwd(const flce_attn* a, const flce_opts* opts) {
  return flce::attention(a, opts, true);
}

size_t flce_attn_sizeof(void) { return sizeof(flce_attn); }

}  // extern "C"
