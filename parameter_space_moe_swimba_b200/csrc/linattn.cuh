// Decay linear attention: what the SIMT and the tensor-core kernels share.
//
// One head's recurrence over a [d_x, d_w] state M, in a form that serves the forward and all three
// gradients ("roles"): a readout stream x, a key stream y, a value stream w,
//   forward:  M = γ M + s_u y_t w_tᵀ;  out_t = s_inter Mᵀ x_t
//   reverse:  G = M + s_u y_t w_tᵀ;    out_t = Gᵀ x_t;  M = γ G             (tokens last to first)
//   o : x = q,  y = k, w = v,  M = S            dq: x = do, y = v,  w = k, M = Sᵀ
//   dv: x = k,  y = q, w = do, M = G, reverse   dk: x = v,  y = do, w = q, M = Gᵀ, reverse
// Between pieces the reverse roles carry M, the adjoint already decayed to the earlier token, so
// that M before the first piece is dL/dS_final itself and M after the last is dL/dS0.
#pragma once

#include "common.cuh"

namespace swimba {

constexpr int kLaChunk = 128;   // tokens per chunk of the tensor-core kernel
constexpr int kLaSimtChunk = 32;  // the fp32 recurrence's segments are whole multiples of this
constexpr int kLaMaxRoles = 3;

// Element (b, t, h, j) of an io tensor: p + b sb + t st + (h / div) d + j, d the role's width.
struct LaStream {
  const void* p;
  int64_t st, sb;
  int div;
};

struct LaRole {
  LaStream x, y, w;
  void* out;             // element (b, t, h, c): out + b out_sb + t out_st + h dw + c
  int64_t out_st, out_sb;
  int out_f32;           // out is fp32 whatever the io type (per-head partials of shared heads)
  int dx, dw;            // rows and columns of M
  int rev;
  float s_inter, s_u;    // the scale belongs to the readout (forward) or to the update (reverse)
  const float* M0;       // element (j, c) of head bh: M0 + bh dx dw + j sj + c sc; or null
  float* M_end;          // likewise
  int sj, sc;
  float* seg;            // [B H, nseg, dx, dw] segment states, or null (one segment)
  int parts;             // bf16 parts of the weighted values, at most: 3 where M itself is an output, else 2
};

struct LaParams {
  LaRole role[kLaMaxRoles];
  int n_roles;
  const float* g;        // log decay per head
  const int32_t* lens;   // or null
  int64_t L;
  int B, H;
  int chunk;             // tokens per chunk: segments are whole chunks
  int nseg, cps;         // segments per sequence, chunks per segment
  int balanced;          // tensor cores: all chunks dealt to the CTAs in equal shares, cutting sequences
  int* hand_flags;       // balanced: per CTA, zeroed before the launch
  float* hand_states;    // balanced: per CTA, the state at the cut of the sequence it begins
  void* status;
};

// γ^e = exp2(lg e) for e >= 0; γ^0 = 1 also for lg = -inf (a head that keeps nothing).
__device__ __forceinline__ float la_pow(float lg, int e) { return e == 0 ? 1.f : exp2f(lg * (float)e); }

// γ^e as hi + lo, for a factor that a state meets again and again: rounded once, a γ near 1 is off by up to 2^-25
// at every use, with the same sign (4096 single tokens at a log decay of -1e-5: 6e-5 of the state; with lo 1e-8).
// A γ^e below e^-1/2 is forgotten within a few uses. lo has hi's sign and is not zero unless γ^e is (or nearly): an
// infinite state then stays what it is.
struct LaDecay {
  float hi, lo;
};
__device__ __forceinline__ LaDecay la_decay(float g, int e) {
  const float x = g * (float)e;
  if (!(fabsf(x) < 0.5f)) {
    const float p = la_pow(g * kLog2e, e);
    return {p, p * 0x1p-40f};
  }
  const float m = expm1f(x), hi = 1.f + m, lo = m - (hi - 1.f);  // exact: |m| < 1
  return lo > 0.f ? LaDecay{hi, lo} : LaDecay{hi - 0x1p-24f, lo + 0x1p-24f};
}

// The j-th of a series of factors for hi + lo, 1/2 < hi <= 1, |lo| <= 2^-24: hi or hi ± 2^-24, whichever keeps the product of all of
// them next to the power. A function of j, so that a series may be taken up anywhere.
__device__ __forceinline__ float la_factor(LaDecay d, int j) {
  const float c = d.lo * 0x1p24f;
  return fmaf(rintf((float)(j + 1) * c) - rintf((float)j * c), 0x1p-24f, d.hi);
}

__device__ __forceinline__ int64_t la_len(const LaParams& p, int b) {
  if (p.lens == nullptr) return p.L;
  const int64_t n = p.lens[b];
  return n < 0 ? 0 : (n > p.L ? p.L : n);
}

// Chunks [c0, c1) of segment `seg`, in natural order (a reverse role walks them from c1 - 1 down and
// counts its segments from the sequence's end).
__device__ __forceinline__ void la_segment(const LaParams& p, int64_t len, int seg, int rev, int& c0, int& c1) {
  const int nch = (int)((uint32_t)(len + p.chunk - 1) / (uint32_t)p.chunk);
  const int a = (int)min((int64_t)nch, (int64_t)seg * p.cps), z = min(nch, a + p.cps);
  c0 = rev ? nch - z : a;
  c1 = rev ? nch - a : z;
}

struct LaPlan {
  bool tc;        // tensor-core kernel (bf16)
  int nseg, cps;  // segments per sequence, chunks per segment
  bool cut;       // sequences may be cut between two CTAs (see run_la_tc): room for the states handed over
};

// Chunks of the longest of `ctas` equal shares of `total` chunks, and 3 for cutting sequences between them.
inline double la_shared_units(int64_t total, int ctas) { return (double)(total / ctas + 3); }

constexpr int kLaCtas = 148;  // one per SM
constexpr size_t kLaHandBytes = (size_t)kLaCtas * 128 * 128 * 4;
constexpr size_t kLaFlagBytes = 1024;

}  // namespace swimba
